"""The operators around the routed experts without a GPU: argument checks of the C ABI
and of the Python binding, and the pins of their oracle."""
import ctypes

import numpy as np
import pytest

from blocks_cases import B, choices, normals, route, sequences
from score_top_expert_gb300 import build as Build

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks
ODD = ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def L():
    Build.build()
    import score_top_expert_gb300.router as r
    return r.lib()


def balance(L, **kw):
    a = dict(x=FAKE, dt=0, idx=FAKE, ld=2, seq=FAKE, T=8, E=16, K=2, S=2, sf=0, loss=FAKE, counts=FAKE,
             stats=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return L.router_balance_loss_fwd(a["x"], a["dt"], a["idx"], a["ld"], a["seq"], a["T"], a["E"],
                                     a["K"], a["S"], a["sf"], 1.0, 0.0, a["loss"], a["counts"],
                                     a["stats"], a["ws"], a["bytes"], None)


SIZES = [(dict(T=-1), -1), (dict(E=0), -1), (dict(K=0), -1), (dict(K=17), -1), (dict(S=0), -1),
         (dict(S=9), -1), (dict(dt=2), -1), (dict(sf=2), -1), (dict(sf=5), -1),
         (dict(seq=None), -1), (dict(T=1 << 20, E=2304), -1), (dict(E=2305), -2),
         (dict(E=64, K=37, ld=37), -2), (dict(stats=None), -1), (dict(stats=ODD), -1),
         (dict(x=None), -1), (dict(counts=None), -1), (dict(T=0, S=2), -1)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(ld=1), -1), (dict(idx=None), -1), (dict(loss=None), -1), (dict(ws=None), -1),
    (dict(ws=ODD), -1), (dict(bytes=64), -1)])
def test_balance_rejects(L, kw, code):
    assert balance(L, **kw) == code


@pytest.mark.parametrize("kw,code", SIZES + [(dict(g=None), -1), (dict(grad=None), -1),
                                             (dict(T=0, S=1), 0)])
def test_balance_bwd_rejects(L, kw, code):
    a = dict(g=FAKE, x=FAKE, dt=0, counts=FAKE, stats=FAKE, seq=FAKE, T=8, E=16, K=2, S=2, sf=0,
             grad=FAKE)
    a.update(kw)
    if a["E"] == 64:
        a.pop("ld")
    assert L.router_balance_loss_bwd(a["g"], a["x"], a["dt"], a["counts"], a["stats"], a["seq"],
                                     a["T"], a["E"], a["K"], a["S"], a["sf"], 1.0, 0.0, a["grad"],
                                     None) == code


def test_balance_workspace(L):
    f = L.router_balance_loss_workspace_bytes
    assert f(-1, 8, 1) == 0 and f(8, 0, 1) == 0 and f(8, 8, 0) == 0 and f(8, 2305, 1) == 0
    assert 0 < f(0, 8, 1) <= f(8192, 8, 1) <= f(8192, 2304, 1) <= f(8192, 2304, 64)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), -1), (dict(D=0), -1), (dict(dt=2), -1), (dict(D=65537), -2), (dict(x=None), -1),
    (dict(q=None), -1), (dict(s=None), -1), (dict(R=0, x=None, q=None, s=None), 0)])
def test_quantize_rejects(L, kw, code):
    a = dict(x=FAKE, dt=1, R=4, D=8, q=FAKE, s=FAKE)
    a.update(kw)
    assert L.router_quantize_rows(a["x"], a["dt"], a["R"], a["D"], a["q"], a["s"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(P=-1), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(D=0), -1), (dict(odt=2), -1),
    (dict(E=2305), -2), (dict(N=65537), -2), (dict(D=65537), -2), (dict(T=-1), -1), (dict(T=0), -1),
    (dict(x=None), -1), (dict(xs=None), -1), (dict(w=None), -1), (dict(ws=None), -1),
    (dict(off=None), -1), (dict(out=None), -1), (dict(P=0, x=None, off=None, out=None), 0)])
def test_w8_rejects(L, kw, code):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, off=FAKE, p2u=FAKE, T=4, P=8, E=4, N=8, D=16, out=FAKE,
             odt=1)
    a.update(kw)
    assert L.router_expert_matmul_w8(a["x"], a["xs"], a["w"], a["ws"], a["off"], a["p2u"], a["T"],
                                     a["P"], a["E"], a["N"], a["D"], a["out"], a["odt"],
                                     None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(K=0), -1), (dict(D=0), -1), (dict(dt=3), -1), (dict(eps=0.0), -1),
    (dict(eps=float("nan")), -1), (dict(K=37, ld=37), -2), (dict(D=8193), -2),
    (dict(T=1 << 30, K=4), -1), (dict(u2p=None), -1), (dict(u2p=None, K=1), -1), (dict(ld=1), -1),
    (dict(kind=3), -1), (dict(kind=-1), -1), (dict(kind=1), -1), (dict(gate=FAKE), -1),
    (dict(z=None), -1), (dict(res=None), -1), (dict(sum=None), -1), (dict(normed=None), -1),
    (dict(rstd=ODD), -1), (dict(T=0, z=None, res=None, sum=None), 0)])
def test_norm_rejects(L, kw, code):
    a = dict(z=FAKE, dt=1, u2p=FAKE, w=FAKE, ld=2, res=FAKE, post=FAKE, gate=None, kind=0, pre=FAKE,
             eps=1e-6, T=4, K=2, D=8, sum=FAKE, normed=FAKE, block=None, rstd=None)
    a.update(kw)
    assert L.router_combine_norm_fwd(a["z"], a["dt"], a["u2p"], a["w"], a["ld"], a["res"], a["post"],
                                     a["gate"], a["kind"], 1.0, a["pre"], a["eps"], a["T"], a["K"],
                                     a["D"], a["sum"], a["normed"], a["block"], a["rstd"],
                                     None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(D=0), -1), (dict(D=8193), -2), (dict(dt=3), -1), (dict(kind=4), -1),
    (dict(gate=FAKE), -1), (dict(gate=FAKE, kind=1), -1), (dict(kind=1, gg=FAKE), -1),
    (dict(gs=None, pre=None), -1), (dict(gn=None), -1), (dict(sum=None), -1), (dict(block=None), -1),
    (dict(rstd=None), -1), (dict(rstd=ODD), -1), (dict(gb=None), -1), (dict(gr=None), -1),
    (dict(gpost=None), -1), (dict(gpre=None), -1), (dict(ws=None), -1), (dict(ws=ODD), -1),
    (dict(bytes=8), -1), (dict(T=0, post=None, pre=None), 0)])
def test_norm_bwd_rejects(L, kw, code):
    a = dict(gs=FAKE, gn=FAKE, dt=1, block=FAKE, sum=FAKE, rstd=FAKE, post=FAKE, gate=None, kind=0,
             pre=FAKE, T=4, D=8, gb=FAKE, gr=FAKE, gg=None, gpost=FAKE, gpre=FAKE, ws=FAKE,
             bytes=1 << 30)
    a.update(kw)
    assert L.router_combine_norm_bwd(a["gs"], a["gn"], a["dt"], a["block"], a["sum"], a["rstd"],
                                     a["post"], a["gate"], a["kind"], 1.0, a["pre"], a["T"], a["D"],
                                     a["gb"], a["gr"], a["gg"], a["gpost"], a["gpre"], a["ws"],
                                     a["bytes"], None) == code


def test_call_shim_returns_the_same_codes(L):
    import score_top_expert_gb300.router as r
    calls = r._calls()
    p = 0x1000
    assert calls.router_quantize_rows(p, 1, -1, 8, p, p, 0) == -1
    assert calls.router_expert_matmul_w8(p, p, p, p, p, p, 4, 8, 4, 8, 65537, p, 1, 0) == -2
    assert calls.router_combine_norm_fwd(p, 1, p, p, 2, p, p, 0, 0, 1.0, p, 0.0, 4, 2, 8, p, p, 0, 0,
                                         0) == -1
    assert calls.router_combine_norm_bwd(p, p, 1, p, p, p, p, 0, 0, 1.0, p, 4, 8193, p, p, 0, p, p, p,
                                         1 << 40, 0) == -2
    assert calls.router_balance_loss_fwd(p, 0, p, 2, p, 8, 16, 2, 2, 0, 1.0, 0.0, p, p, p, p, 8,
                                         0) == -1
    assert calls.router_balance_loss_bwd(p, p, 0, p, p, p, 8, 2305, 2, 2, 0, 1.0, 0.0, p, 0) == -2


def test_binding_refuses_host_tensors(L):
    torch = pytest.importorskip("torch")
    import score_top_expert_gb300.router as r
    rows = torch.zeros(4, 8)
    for call in (lambda: r.router_quantize_rows(rows),
                 lambda: r.router_expert_matmul_w8(rows.char(), rows[:, 0], rows.char()[None],
                                                   rows[:1], torch.zeros(2, dtype=torch.int32)),
                 lambda: r.router_combine_norm_fwd(rows, rows),
                 lambda: r.router_combine_norm_bwd(rows, None, None, None, None),
                 lambda: r.router_balance_loss_fwd(rows, torch.zeros(4, 2, dtype=torch.int32)),
                 lambda: r.router_balance_loss_bwd(rows[0, :2], rows, rows.int(), rows, 2)):
        with pytest.raises(ValueError):
            call()


# ---- the oracle's pins --------------------------------------------------------------------
def test_balance_oracle_of_even_choices():
    # every expert chosen equally and equal logits: the loss is coeff, the gradient zero
    idx = np.array([[0, 1], [2, 3], [1, 0], [3, 2]], np.int32)
    for score in ("softmax", "sigmoid"):
        loss, counts = B.balance_loss(np.zeros((4, 4)), idx, score, 0.25, 0.0)
        assert loss[0] == pytest.approx(0.25, rel=1e-14) and counts.tolist() == [[2, 2, 2, 2]]
        grad, _ = B.balance_loss_bwd([1.0, 0.0], np.zeros((4, 4)), counts, 2, score, 0.25, 0.0)
        assert np.abs(grad).max() <= 1e-17
    # two sequences of one expert each: E times their share, averaged; ln 2 squared for z
    loss, counts = B.balance_loss(np.zeros((3, 2)), np.array([[0], [1], [1]]), "softmax", 1.0, 3.0,
                                  [0, 1, 3])
    assert loss[0] == pytest.approx(1.0) and loss[1] == pytest.approx(3.0 * np.log(2.0) ** 2)
    assert counts.tolist() == [[1, 0], [0, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_oracle_gradient_against_differences(score):
    T, E, K = 7, 6, 2
    x, idx = normals((T, E), 1, "f32").astype(np.float64), choices(T, E, K, 2, drop=0.2)
    seq = sequences(T, 3, 1, 3)
    _, counts = B.balance_loss(x, idx, score, 0.7, 0.3, seq)
    grad, mag = B.balance_loss_bwd([2.0, 5.0], x, counts, K, score, 0.7, 0.3, seq)
    step = 1e-6
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(x)
            d[t, e] = step
            up, down = (B.balance_loss(x + s * d, idx, score, 0.7, 0.3, seq)[0] for s in (1, -1))
            assert abs(np.dot([2.0, 5.0], up - down) / (2 * step) - grad[t, e]) <= 1e-8
    assert np.all(np.abs(grad) <= mag + 1e-12) and not grad[T - 1].any()


def test_quantize_oracle():
    q, s = B.quantize_rows([[1.0, -127.0, 0.5, 2.5, 3.5], [0.0] * 5, [254.0, 1.0, 3.0, -1.0, 5.0]])
    assert s.tolist() == [1.0, 0.0, 2.0]
    assert q.tolist() == [[1, -127, 0, 2, 4], [0] * 5, [127, 0, 2, 0, 2]]


def test_w8_oracle_by_loops():
    T, E, K, N, D = 5, 3, 2, 4, 6
    m = route(T, E, K, 1, drop=0.2)
    rng = np.random.default_rng(2)
    x, w = rng.integers(-128, 128, (T, D)), rng.integers(-128, 128, (E, N, D))
    xs, ws = rng.random(T), rng.random((E, N))
    got, mag = B.expert_matmul_w8(x, xs, w, ws, m["off"], m["p2u"], T)
    for e in range(E):
        for p in range(m["off"][e], m["off"][e + 1]):
            t = m["p2u"][p] % T
            for n in range(N):
                want = sum(int(x[t, d]) * int(w[e, n, d]) for d in range(D)) * xs[t] * ws[e, n]
                assert got[p, n] == pytest.approx(want, rel=1e-13, abs=1e-13)
    assert np.isnan(got[m["off"][-1]:]).all()
    assert np.all(np.abs(got[:m["off"][-1]]) <= mag[:m["off"][-1]] + 1e-9)


def test_norm_oracle_by_hand():
    r = B.combine_norm_fwd([[3.0, 4.0]], [[1.0, -1.0]], post_weight=[1.0, 2.0], gate=[0.5],
                           residual_scale=2.0, pre_weight=[1.0, 10.0], eps=12.5)
    # mean of squares 12.5, with eps 25: a fifth
    assert r["rstd"][0, 0] == pytest.approx(0.2) and r["x"][0] == pytest.approx([1.6, 0.6])
    assert r["normed"][0] == pytest.approx(np.array([1.6, 6.0]) / np.sqrt(1.46 + 12.5))


@pytest.mark.parametrize("gate", ["none", "token", "value"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_norm_oracle_gradient_against_differences(gate, post, pre):
    T, D = 3, 5
    rng = np.random.default_rng(4)
    a = {"y": rng.standard_normal((T, D)), "res": rng.standard_normal((T, D)),
         "gate": {"none": None, "token": rng.random(T), "value": rng.random((T, D))}[gate],
         "post": rng.random(D) + 0.5 if post else None, "pre": rng.random(D) + 0.5 if pre else None}
    gs, gn = rng.standard_normal((T, D)), rng.standard_normal((T, D))

    def forward(d):
        return B.combine_norm_fwd(d["y"], d["res"], None, None, d["post"], d["gate"], 0.5, d["pre"])

    def value(d):
        r = forward(d)
        return (r["x"] * gs).sum() + ((r["normed"] * gn).sum() if pre else 0.0)

    r = forward(a)
    got = B.combine_norm_bwd(gs, gn if pre else None, r["y"], r["x"], r["rstd"], a["post"], a["gate"],
                             0.5, a["pre"])
    for name, key in (("grad_block", "y"), ("grad_residual", "res"), ("grad_gate", "gate"),
                      ("grad_post_weight", "post"), ("grad_pre_weight", "pre")):
        if a[key] is None:
            assert name not in got
            continue
        grad, mag = got[name]
        for i in np.ndindex(a[key].shape):
            d = np.zeros_like(a[key])
            d[i] = 1e-6
            diff = (value(a | {key: a[key] + d}) - value(a | {key: a[key] - d})) / 2e-6
            assert abs(diff - grad[i]) <= 1e-8 * max(1.0, abs(grad[i]))
        assert np.all(np.abs(grad) <= mag * (1 + 1e-12))
