"""The experts' products, their gradients, the 4-bit products and the weighted
combination against the float64 oracle, and a whole expert layer."""
import numpy as np
import pytest

from experts_cases import X, assert_within, normals, route, tolerance, w4_weights

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def R():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from score_top_expert_gb300 import build
    build.build()
    import score_top_expert_gb300.router as r
    r.lib()
    return r


def up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(DT[dtype])


def down(t):
    return t.detach().double().cpu().numpy()


def counts(m):
    return np.diff(m["off"].astype(np.int64))


def check_product(R, m, T, E, K, N, D, dtype, out, gather, seed=1):
    """Forward and both gradients of one product; rows no expert owns keep a mark."""
    P = T * K
    placed = int(m["off"][-1])
    x = normals((T if gather else P, D), seed, dtype)
    w = normals((E, N, D), seed + 1, dtype, D ** -0.5)
    g = normals((P, N), seed + 2, dtype)
    p2u = m["p2u"] if gather else None
    xd, wd, gd, off = up(x, dtype), up(w, dtype), up(g, dtype), up(m["off"])
    pd = None if p2u is None else up(p2u)
    mark = 77.0

    y = torch.full((P, N), mark, dtype=DT[out], device=DEV)
    R.router_expert_matmul(xd, wd, off, pd, out=y, out_dtype=DT[out])
    gx = torch.full((P, D), mark, dtype=DT[out], device=DEV)
    R.router_expert_matmul_bwd_input(gd, wd, off, grad_x=gx, out_dtype=DT[out])
    gw = torch.full((E, N, D), mark, dtype=DT[out], device=DEV)
    R.router_expert_matmul_bwd_weight(gd, xd, off, pd, grad_weight=gw, out_dtype=DT[out])
    torch.cuda.synchronize()
    assert R.device_status() == 0

    ref, mag = X.expert_matmul(x, w, m["off"], p2u, T)
    assert_within(down(y)[:placed], ref[:placed], tolerance(ref, mag, D, out)[:placed], "out")
    assert (down(y)[placed:] == mark).all()
    ref, mag = X.expert_matmul_bwd_input(g, w, m["off"])
    assert_within(down(gx)[:placed], ref[:placed], tolerance(ref, mag, N, out)[:placed], "grad_x")
    assert (down(gx)[placed:] == mark).all()
    ref, mag = X.expert_matmul_bwd_weight(g, x, m["off"], p2u, T)
    length = counts(m)[:, None, None]
    assert_within(down(gw), ref, tolerance(ref, mag, length, out), "grad_weight")


# sizes: whole tiles, one value, odd and unaligned rows, one row of many tiles
PRODUCTS = [
    (64, 8, 2, 128, 64, "bf16", "bf16", True), (64, 8, 2, 128, 64, "bf16", "f32", False),
    (1, 4, 1, 8, 8, "bf16", "bf16", True), (1, 64, 4, 1024, 1024, "bf16", "bf16", True),
    (1, 1, 1, 1, 1, "bf16", "f32", True), (3, 5, 5, 33, 17, "bf16", "bf16", True),
    (37, 7, 3, 200, 136, "bf16", "f32", True), (37, 7, 3, 136, 200, "bf16", "bf16", False),
    (301, 3, 2, 264, 72, "bf16", "f32", True), (700, 2, 1, 520, 1000, "bf16", "bf16", True),
    (1100, 1, 1, 136, 264, "bf16", "f32", True), (129, 16, 4, 320, 328, "bf16", "bf16", False),
    (70, 300, 6, 24, 40, "bf16", "f32", True), (50, 2304, 36, 16, 32, "bf16", "bf16", True),
    (515, 4, 2, 257, 255, "bf16", "bf16", True), (40, 6, 2, 64, 65, "bf16", "f32", True),
    (40, 6, 2, 65, 64, "bf16", "f32", True),
    # many experts of unequal sizes, taken by size
    (3000, 40, 3, 264, 72, "bf16", "f32", True), (9000, 150, 2, 72, 136, "bf16", "bf16", False),
    # contractions and experts longer than a fp32 output's segment
    (900, 2, 1, 1000, 1608, "bf16", "f32", True), (20, 8, 2, 1600, 1608, "bf16", "f32", False),
    (1700, 1, 1, 264, 72, "bf16", "f32", True), (1700, 1, 1, 264, 72, "bf16", "bf16", True),
    (64, 8, 2, 128, 64, "f32", "f32", True), (37, 7, 3, 67, 129, "f32", "f32", True),
    (20, 4, 2, 1100, 1301, "f32", "f32", True), (1100, 1, 1, 40, 33, "f32", "f32", True),
    (30, 4, 2, 1003, 1201, "bf16", "f32", True), (260, 2, 1, 129, 130, "bf16", "bf16", False),
    (3, 9, 4, 600, 776, "bf16", "bf16", True), (4, 9, 9, 40, 520, "bf16", "f32", False),
    (5, 3, 2, 33, 515, "f32", "bf16", False), (300, 2, 2, 100, 60, "f32", "f32", True),
]


@pytest.mark.parametrize("T,E,K,N,D,dtype,out,gather", PRODUCTS)
def test_products(R, T, E, K, N, D, dtype, out, gather):
    check_product(R, route(T, E, K, seed=T + E + K), T, E, K, N, D, dtype, out, gather)


@pytest.mark.parametrize("dtype,gather", [("bf16", True), ("bf16", False), ("f32", True)])
def test_products_with_empty_experts_and_skipped_choices(R, dtype, gather):
    m = route(90, 12, 3, seed=5, drop=0.3, empty=(0, 4, 5, 11))
    assert (counts(m) == 0).sum() >= 4 and m["off"][-1] < 270
    check_product(R, m, 90, 12, 3, 72, 136, dtype, "f32", gather)


def test_products_when_every_choice_is_skipped(R):
    m = route(20, 6, 2, seed=6, drop=1.1)
    assert m["off"][-1] == 0
    check_product(R, m, 20, 6, 2, 64, 64, "bf16", "bf16", True)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 513])
def test_products_around_the_tile_sizes(R, rows):
    # two experts: one with exactly ``rows`` rows, one with three
    T = rows + 3
    idx = np.array([0] * rows + [1] * 3, np.int32)
    m = dict(off=np.array([0, rows, T], np.int32), p2u=np.arange(T, dtype=np.int32), idx=idx)
    check_product(R, m, T, 2, 1, 136, 72, "bf16", "f32", True, seed=rows)


def test_a_nan_stays_in_its_rows_and_expert(R):
    T, E, K, N, D = 40, 4, 2, 72, 136
    m = route(T, E, K, seed=8)
    x = normals((T, D), 1, "bf16")
    w = normals((E, N, D), 2, "bf16", 0.1)
    g = normals((T * K, N), 3, "bf16")
    x[7, 5] = np.nan
    x[9, 6] = np.inf
    e0 = int(m["idx"][7, 0])
    off, p2u = up(m["off"]), up(m["p2u"])
    y = down(R.router_expert_matmul(up(x, "bf16"), up(w, "bf16"), off, p2u))
    bad = np.isin(m["p2u"] % T, [7, 9])
    assert np.isfinite(y[~bad]).all() and not np.isfinite(y[bad]).any()
    gw = down(R.router_expert_matmul_bwd_weight(up(g, "bf16"), up(x, "bf16"), off, p2u))
    touched = np.unique(m["idx"][[7, 9]])
    for e in range(E):
        cols = np.zeros(D, bool)
        if e in m["idx"][7]:
            cols[5] = True
        if e in m["idx"][9]:
            cols[6] = True
        assert np.isfinite(gw[e][:, ~cols]).all(), e
        assert not np.isfinite(gw[e][:, cols]).any(), e
    assert e0 in touched
    g[0, 3] = np.nan  # the first expert with rows only
    first = int(np.nonzero(counts(m))[0][0])
    x = normals((T, D), 1, "bf16")
    gx = down(R.router_expert_matmul_bwd_input(up(g, "bf16"), up(w, "bf16"), off))
    assert np.isnan(gx[0]).all() and np.isfinite(gx[1:]).all()
    gw = down(R.router_expert_matmul_bwd_weight(up(g, "bf16"), up(x, "bf16"), off, p2u))
    assert np.isnan(gw[first][3]).all()
    gw[first][3] = 0
    assert np.isfinite(gw).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 136), ("bf16", 135), ("f32", 136)])
def test_a_nan_among_rows_in_order_stays_there(R, dtype, D):
    # rows in order are brought in whole boxes that may reach into the next expert
    E, N = 3, 72
    off = np.array([0, 40, 45, 100], np.int32)
    x, w = normals((100, D), 1, dtype), normals((E, N, D), 2, dtype, 0.1)
    g = normals((100, N), 3, dtype)
    x[42] = np.nan
    y = down(R.router_expert_matmul(up(x, dtype), up(w, dtype), up(off)))
    bad = np.arange(100) == 42
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()
    gw = down(R.router_expert_matmul_bwd_weight(up(g, dtype), up(x, dtype), up(off)))
    assert np.isnan(gw[1]).all() and np.isfinite(gw[[0, 2]]).all()
    x = normals((100, D), 1, dtype)
    g[44] = np.inf
    gw = down(R.router_expert_matmul_bwd_weight(up(g, dtype), up(x, dtype), up(off)))
    assert not np.isfinite(gw[1]).any() and np.isfinite(gw[[0, 2]]).all()
    gx = down(R.router_expert_matmul_bwd_input(up(g, dtype), up(w, dtype), up(off)))
    bad = np.arange(100) == 44
    assert not np.isfinite(gx[bad]).any() and np.isfinite(gx[~bad]).all()


def test_empty_batches(R):
    w = torch.randn(3, 8, 16, device=DEV).bfloat16()
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 16, device=DEV, dtype=torch.bfloat16)
    g = torch.empty(0, 8, device=DEV, dtype=torch.bfloat16)
    p2u = torch.empty(0, dtype=torch.int32, device=DEV)
    assert R.router_expert_matmul(x, w, off, p2u).shape == (0, 8)
    assert R.router_expert_matmul_bwd_input(g, w, off).shape == (0, 16)
    gw = R.router_expert_matmul_bwd_weight(g, x, off, p2u)
    assert gw.shape == (3, 8, 16) and (gw == 0).all()
    assert R.router_combine_fwd(x, p2u, 2).shape == (0, 16)
    gz, gwt = R.router_combine_bwd(x, p2u, 2, x)
    assert gz.shape == (0, 16) and gwt.shape == (0, 2)
    q = torch.zeros(3, 8, 16, dtype=torch.uint8, device=DEV)
    s = torch.ones(3, 8, 1, device=DEV).bfloat16()
    x = torch.empty(0, 32, device=DEV, dtype=torch.bfloat16)
    assert R.router_expert_matmul_w4(x, q, s, off, p2u).shape == (0, 8)


def test_strided_inputs_and_column_views(R):
    T, E, K, N, D = 33, 6, 2, 64, 72
    m = route(T, E, K, seed=11)
    off, p2u, u2p = up(m["off"]), up(m["p2u"]), up(m["u2p"])
    wide = up(normals((T, 2 * D), 1, "bf16"), "bf16")
    w = up(normals((E, N, D), 2, "bf16", 0.1), "bf16")
    y = R.router_expert_matmul(wide[:, D:], w, off, p2u)
    assert torch.equal(y, R.router_expert_matmul(wide[:, D:].contiguous(), w, off, p2u))
    odd = torch.empty(T * D + 1, device=DEV, dtype=torch.bfloat16)[1:].view(T, D)  # 2-byte aligned
    odd.copy_(wide[:, D:])
    assert_within(down(R.router_expert_matmul(odd, w, off, p2u, out_dtype=torch.float32)),
                  *tolerances_of(X.expert_matmul(down(odd), down(w), m["off"], m["p2u"], T), D))
    tw = up(np.concatenate([m["w"], m["w"]], 1))[:, :K]  # a column view of the weights
    z = R.router_combine_fwd(y, u2p, K, tw)
    assert torch.equal(z, R.router_combine_fwd(y, u2p, K, tw.contiguous()))
    with pytest.raises(ValueError, match="contiguous"):
        R.router_expert_matmul(wide[:, D:], w.transpose(1, 2).contiguous().transpose(1, 2), off, p2u)


def tolerances_of(ref_mag, length, out="f32"):
    ref, mag = ref_mag
    return ref, tolerance(ref, mag, length, out)


def test_weights_past_32_bit_offsets(R):
    # 40 x 8192 x 8192 elements: the last expert's weights lie behind 2^31 elements
    E, N, D, T = 40, 8192, 8192, 9
    assert (E - 1) * N * D > 2 ** 31
    try:
        w = torch.zeros(E, N, D, dtype=torch.bfloat16, device=DEV)
        last = up(normals((N, D), 1, "bf16", 0.01), "bf16")
        w[E - 1] = last
        x = up(normals((T, D), 2, "bf16"), "bf16")
        off = torch.full((E + 1,), 0, dtype=torch.int32, device=DEV)
        off[E] = T
        p2u = torch.arange(T, dtype=torch.int32, device=DEV)
        y = R.router_expert_matmul(x, w, off, p2u, out_dtype=torch.float32)
        xr, lr = x.double(), last.double()
        ref, mag = down(xr @ lr.t()), down(xr.abs() @ lr.abs().t())
        assert_within(down(y), ref, tolerance(ref, mag, D, "f32"), "out")
        g = up(normals((T, N), 3, "bf16"), "bf16")
        gx = R.router_expert_matmul_bwd_input(g, w, off, out_dtype=torch.float32)
        ref, mag = down(g.double() @ lr), down(g.double().abs() @ lr.abs())
        assert_within(down(gx), ref, tolerance(ref, mag, N, "f32"), "grad_x")
        gw = R.router_expert_matmul_bwd_weight(g, x, off, p2u, grad_weight=w)
        ref = g.double().t() @ xr
        assert_within(down(gw[E - 1]), down(ref),
                      tolerance(down(ref), down(g.double().abs().t() @ xr.abs()), T, "bf16"), "gw")
        assert not gw[:E - 1].any()
    finally:
        torch.cuda.empty_cache()


# ---- 4-bit weights -----------------------------------------------------------
@pytest.mark.parametrize("T,E,K,N,D,group,zeros,out,gather", [
    (1, 8, 2, 64, 128, 128, False, "bf16", True), (1, 4, 1, 1, 32, 32, True, "f32", True),
    (4, 16, 3, 40, 96, 32, True, "f32", True), (7, 5, 5, 17, 320, 64, False, "f32", False),
    (33, 6, 2, 100, 256, 128, True, "bf16", True), (64, 3, 2, 130, 1056, 32, False, "f32", True),
    (9, 300, 6, 24, 64, 64, True, "f32", True), (200, 2, 1, 48, 640, 128, False, "bf16", True),
    (3, 4, 2, 40, 8224, 32, True, "f32", True), (9, 3, 2, 20, 4480, 128, True, "bf16", False),
    (2, 2304, 36, 16, 2176, 128, True, "f32", True), (64, 2304, 36, 8, 32, 32, False, "bf16", True),
])
def test_w4(R, T, E, K, N, D, group, zeros, out, gather):
    m = route(T, E, K, seed=T + E + N)
    x = normals((T if gather else T * K, D), 3, "bf16")
    q, s, z = w4_weights(E, N, D, group, zeros, 4)
    p2u = m["p2u"] if gather else None
    y = R.router_expert_matmul_w4(up(x, "bf16"), up(q), up(s, "bf16"), up(m["off"]),
                                  None if p2u is None else up(p2u),
                                  zeros=None if z is None else up(z), out_dtype=DT[out])
    ref, mag = X.expert_matmul_w4(x, q, s, z, group, m["off"], p2u, T)
    # the scaling of each group's sum is one more rounding per product
    assert_within(down(y), ref, tolerance(ref, mag, 2 * D, out), "out")


def test_w4_with_empty_experts_and_skipped_choices(R):
    T, E, K, N, D = 21, 9, 3, 33, 192
    m = route(T, E, K, seed=3, drop=0.4, empty=(0, 8))
    placed = int(m["off"][-1])
    x = normals((T, D), 3, "bf16")
    x[T - 1] = np.nan  # a token's NaN stays in its own rows
    q, s, z = w4_weights(E, N, D, 64, True, 4)
    y = torch.full((T * K, N), 5.0, device=DEV)
    R.router_expert_matmul_w4(up(x, "bf16"), up(q), up(s, "bf16"), up(m["off"]), up(m["p2u"]),
                              zeros=up(z), out=y, out_dtype=torch.float32)
    assert (down(y)[placed:] == 5.0).all()
    ref, mag = X.expert_matmul_w4(x, q, s, z, 64, m["off"], m["p2u"], T)
    keep = (m["p2u"][:placed] % T) != T - 1
    assert_within(down(y)[:placed][keep], ref[:placed][keep],
                  tolerance(ref, mag, 2 * D, "f32")[:placed][keep], "out")
    assert np.isnan(down(y)[:placed][~keep]).all()


def test_w4_long_rows_over_many_tasks(R):
    # more tiles than warps share, and activations longer than one staged panel
    E, K, T, N, D, group = 8, 2, 8, 9984, 4224, 128
    m = route(T, E, K, seed=7)
    gen = torch.Generator(device=DEV).manual_seed(3)
    try:
        q = torch.randint(0, 256, (E, N, D // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s = (torch.rand(E, N, D // group, generator=gen, device=DEV) * 0.01).bfloat16()
        z = torch.randint(0, 16, (E, N, D // group), generator=gen, device=DEV, dtype=torch.uint8)
        x = torch.randn(T, D, generator=gen, device=DEV).bfloat16()
        y = R.router_expert_matmul_w4(x, q, s, up(m["off"]), up(m["p2u"]), zeros=z,
                                      out_dtype=torch.float32)
        for e in range(E):
            a, b = int(m["off"][e]), int(m["off"][e + 1])
            if a == b:
                continue
            w = torch.stack((q[e] & 15, q[e] >> 4), 2).view(N, D // group, group).double()
            w = ((w - z[e].double()[..., None]) * s[e].double()[..., None]).view(N, D)
            xe = x[torch.from_numpy(m["p2u"][a:b] % T).long().to(DEV)].double()
            ref, mag = down(xe @ w.t()), down(xe.abs() @ w.abs().t())
            assert_within(down(y[a:b]), ref, tolerance(ref, mag, 2 * D, "f32"), f"expert {e}")
    finally:
        torch.cuda.empty_cache()


# ---- combination ---------------------------------------------------------------
@pytest.mark.parametrize("T,E,K,D,dtype,weighted", [
    (1, 8, 8, 2048, "bf16", True), (1, 1, 1, 1, "f32", False), (33, 40, 36, 72, "bf16", True),
    (64, 16, 5, 515, "f32", True), (50, 9, 4, 1000, "f32", True), (50, 9, 4, 1001, "bf16", False),
    (7, 64, 33, 8, "f32", True), (300, 12, 2, 4104, "bf16", True), (40, 12, 32, 4100, "f32", False),
])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_combine(R, T, E, K, D, dtype, weighted, drop):
    E = max(E, K)
    m = route(T, E, K, seed=T + D, drop=drop)
    z = normals((T * K, D), 1, dtype)
    g = normals((T, D), 2, dtype)
    w = m["w"] if weighted else None
    zd, gd, u2p = up(z, dtype), up(g, dtype), up(m["u2p"])
    if drop:  # rows that no choice names are never read
        zd[int(m["off"][-1]):] = float("nan")
    wd = None if w is None else up(w)
    y = R.router_combine_fwd(zd, u2p, K, wd)
    ref, mag = X.combine_fwd(z, m["u2p"], K, w)
    assert_within(down(y), ref, tolerance(ref, mag, K, dtype), "out")
    gz = torch.full((T * K, D), 3.0, dtype=DT[dtype], device=DEV)
    gz, gw = R.router_combine_bwd(gd, u2p, K, zd, wd, grad_expert_out=gz)
    rz, rw, mag = X.combine_bwd(g, m["u2p"], K, z, w)
    named = ~np.isnan(rz[:, 0])
    assert_within(down(gz)[named], rz[named],
                  tolerance(rz[named], np.abs(rz[named]), 1, dtype), "grad_expert_out")
    assert (down(gz)[~named] == 3.0).all()
    assert_within(down(gw), rw, tolerance(rw, mag, D, "f32"), "grad_weights")
    gz2, none = R.router_combine_bwd(gd, u2p, K, None, wd, grad_expert_out=torch.full_like(gz, 3.0))
    assert none is None and torch.equal(gz, gz2)


def test_combine_unaligned_rows_and_wild_map_entries(R):
    T, K, D = 9, 2, 24
    z = torch.empty(T * K * D + 1, device=DEV)[1:].view(T * K, D)  # 4-byte aligned rows
    z.copy_(up(normals((T * K, D), 1, "f32")))
    u2p = np.random.default_rng(2).permutation(T * K).astype(np.int32)
    u2p[[1, 4, 7]] = [T * K, 2 ** 31 - 1, -(2 ** 31)]  # outside: no choice
    y = R.router_combine_fwd(z, up(u2p), K)
    ref, mag = X.combine_fwd(down(z), u2p, K)
    assert_within(down(y), ref, tolerance(ref, mag, K, "f32"))
    g = up(normals((T, D), 3, "f32"))
    gz, gw = R.router_combine_bwd(g, up(u2p), K, z)
    rz, rw, mag = X.combine_bwd(down(g), u2p, K, down(z))
    named = ~np.isnan(rz[:, 0])
    assert np.array_equal(down(gz)[named], rz[named])
    assert_within(down(gw), rw, tolerance(rw, mag, D, "f32"))


def test_wild_offsets_stay_inside_the_buffers(R):
    # offsets out of range and out of order are clamped: rows of each clamped
    # range are computed, the marks around the buffers survive
    E, P, N, D = 5, 40, 64, 64
    off = up(np.array([-5, 10, 4, 30, 1000, 2 ** 31 - 1], np.int32))
    buf = torch.full((P + 20, N), 9.0, device=DEV)
    w = up(normals((E, N, D), 1, "bf16", 0.1), "bf16")
    x = up(normals((P, D), 2, "bf16"), "bf16")
    R.router_expert_matmul(x, w, off, out=buf[10:P + 10], out_dtype=torch.float32)
    assert (buf[:10] == 9.0).all() and (buf[P + 10:] == 9.0).all()
    xd, wd = down(x), down(w)
    got = down(buf[10:P + 10])
    ref, mag = xd[30:40] @ wd[3].T, np.abs(xd[30:40]) @ np.abs(wd[3]).T
    assert_within(got[30:40], ref, tolerance(ref, mag, D, "f32"))
    gw = R.router_expert_matmul_bwd_weight(up(normals((P, N), 3, "bf16"), "bf16"), x, off)
    assert torch.isfinite(gw).all()


# ---- the operators together ------------------------------------------------------
def layer(R, x, w1, w2, logits, K, sf):
    """Router, experts and combination; what the backward needs beside it."""
    tw, idx, *_ = R.router_topk_fwd_compact(logits, K, sf)
    off, p2u, u2p, _ = R.router_expert_maps(idx, logits.shape[1])
    h = R.router_expert_matmul(x, w1, off, p2u)
    a, b = h.float().chunk(2, dim=1)
    act = (torch.nn.functional.silu(a) * b).to(h.dtype)
    z = R.router_expert_matmul(act, w2, off)
    return R.router_combine_fwd(z, u2p, K, tw), (tw, idx, off, p2u, u2p, h, act, z)


@pytest.mark.parametrize("T,E,K,D,F,dtype", [(50, 16, 4, 72, 40, "bf16"), (200, 8, 2, 264, 136, "bf16"),
                                             (31, 12, 3, 33, 21, "f32")])
def test_expert_layer_and_its_gradients(R, T, E, K, D, F, dtype):
    x = up(normals((T, D), 1, dtype), dtype)
    w1 = up(normals((E, 2 * F, D), 2, dtype, D ** -0.5), dtype)
    w2 = up(normals((E, D, F), 3, dtype, F ** -0.5), dtype)
    logits = up(normals((T, E), 4, "f32"))
    gy = up(normals((T, D), 5, dtype), dtype)
    y, (tw, idx, off, p2u, u2p, h, act, z) = layer(R, x, w1, w2, logits, K, "softmax_post")

    gz, gtw = R.router_combine_bwd(gy, u2p, K, z, tw)
    gw2 = R.router_expert_matmul_bwd_weight(gz, act, off, out_dtype=torch.float32)
    gact = R.router_expert_matmul_bwd_input(gz, w2, off)
    hd = h.double().requires_grad_()
    a, b = hd.chunk(2, dim=1)
    (torch.nn.functional.silu(a) * b).backward(gact.double())
    gh = hd.grad.to(h.dtype)
    gw1 = R.router_expert_matmul_bwd_weight(gh, x, off, p2u, out_dtype=torch.float32)
    gx = R.router_combine_fwd(R.router_expert_matmul_bwd_input(gh, w1, off), u2p, K)

    # the same layer in float64 by autograd, on the same choices
    leaves = [t.double().cpu().requires_grad_() for t in (x, w1, w2, tw)]
    X64, W1, W2, TW = leaves
    out = torch.zeros(T, D, dtype=torch.float64)
    rows = []
    ch = idx.cpu().long()
    for t in range(T):
        acc = 0
        for k in range(K):
            hh = W1[ch[t, k]] @ X64[t]
            acc = acc + TW[t, k] * (W2[ch[t, k]] @ (torch.nn.functional.silu(hh[:F]) * hh[F:]))
        rows.append(acc)
    out = torch.stack(rows)
    out.backward(gy.double().cpu())

    # chained roundings: h, act, z and y (forward), gz, gact, gh, grad_x rows and
    # their sum (backward) are each off by half a step of their own size
    step = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[dtype]

    def close(got, ref, roundings, what):
        got, ref = got.double().cpu(), ref.detach()
        rel = float((got - ref).norm() / ref.norm())
        # in the 2-norm independent roundings add at most linearly; a product
        # spreads an operand's relative error without raising it beyond its
        # condition here (random operands: norms of sums of squares), fp32 sums
        # of a few hundred products add 2^-20
        assert rel <= roundings * step + 2.0 ** -20, (what, rel)

    close(y, out, 4, "y")
    close(gx, X64.grad, 6, "grad_x")
    close(gw1, W1.grad, 5, "grad_w1")
    close(gw2, W2.grad, 4, "grad_w2")
    close(gtw, TW.grad, 4, "grad_topk_weights")


def test_calls_repeat_bit_for_bit_and_replay_from_a_graph(R):
    T, E, K, D, F = 96, 32, 4, 136, 72
    w1 = up(normals((E, 2 * F, D), 2, "bf16", 0.1), "bf16")
    w2 = up(normals((E, D, F), 3, "bf16", 0.1), "bf16")
    xs = [up(normals((T, D), s, "bf16"), "bf16") for s in (5, 6, 7)]
    ls = [up(normals((T, E), s, "f32")) for s in (8, 9, 10)]
    gys = [up(normals((T, D), s, "bf16"), "bf16") for s in (11, 12, 13)]
    x, logits, gy = xs[0].clone(), ls[0].clone(), gys[0].clone()

    def step():
        y, (tw, idx, off, p2u, u2p, h, act, z) = layer(R, x, w1, w2, logits, K, "softmax")
        gz, gtw = R.router_combine_bwd(gy, u2p, K, z, tw)
        gw2 = R.router_expert_matmul_bwd_weight(gz, act, off)
        gact = R.router_expert_matmul_bwd_input(gz, w2, off)
        return y, gtw, gw2, gact

    eager = []
    for i in range(3):
        x.copy_(xs[i]); logits.copy_(ls[i]); gy.copy_(gys[i])
        first = [t.clone() for t in step()]
        again = step()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        eager.append(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in (2, 0, 1):
        x.copy_(xs[i]); logits.copy_(ls[i]); gy.copy_(gys[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager[i]))


@pytest.mark.parametrize("T,dtype", [(300, "bf16"), (300, "f32"), (6, "bf16")])
def test_two_streams_at_once(R, T, dtype):
    E, K, N, D = 16, 4, 264, 520
    m = route(T, E, K, seed=4)
    off, p2u = up(m["off"]), up(m["p2u"])
    w = up(normals((E, N, D), 2, dtype, 0.1), dtype)
    xs = [up(normals((T, D), s, dtype), dtype) for s in (1, 2)]
    refs = [R.router_expert_matmul(x, w, off, p2u) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(R.router_expert_matmul(xs[i], w, off, p2u))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, refs[i]) for o in outs[i])
