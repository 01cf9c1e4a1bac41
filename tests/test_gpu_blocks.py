"""The sequence-wise balance loss, the row quantisation, the 8-bit products and the
norms around an expert block against the float64 oracle, and a run of them together."""
import numpy as np
import pytest

from blocks_cases import (B, HALF_STEP, O, STEP, assert_within, balance_loss_tolerance, choices,
                          norm_grad_tolerance, norm_tolerances, normals, route, score_error,
                          sequences)

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
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(DT[dtype])


def down(t):
    return t.detach().double().cpu().numpy()


def shifted(t, by):
    """The same contiguous tensor, ``by`` elements behind an aligned address."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)[by:]
    return flat.view(t.shape).copy_(t)


# ---- balance loss -------------------------------------------------------------------
def check_balance(R, T, E, K, seq, score, z, dtype, seed, scale=1.0, drop=0.0, off=0):
    x = normals((T, E), seed, dtype, scale)
    idx = choices(T, E, K, seed + 1, drop)
    g = np.array([0.7, 1.3], np.float32)
    xd, id_, sd = up(x, dtype), up(idx), up(seq)
    if off:
        xd = shifted(xd, off)
    loss, counts, stats = R.router_balance_loss_fwd(xd, id_, score, 0.01, z, sd)
    grad = torch.full((T, E), 77.0, dtype=DT[dtype], device=DEV)
    if off:
        grad = shifted(grad, off)
    R.router_balance_loss_bwd(up(g), xd, counts, stats, K, score, 0.01, z, sd, grad_logits=grad)
    torch.cuda.synchronize()
    f = np.float64(np.float32(0.01)), np.float64(np.float32(z))
    ref, ref_counts = B.balance_loss(x, idx, score, *f, seq)
    assert np.array_equal(counts.cpu().numpy(), ref_counts)
    assert_within(down(loss), ref, balance_loss_tolerance(x.astype(np.float64), score, ref), "loss")
    ref, mag = B.balance_loss_bwd(g, x, ref_counts, K, score, *f, seq)
    # products of the score (twice in the sum), the row's sum and a few factors
    tol = (2 * score_error(x, score) + score_error(x, "softmax") + 48 * STEP) * mag
    assert_within(down(grad), ref, tol + HALF_STEP[dtype] * (np.abs(ref) + tol) + 1e-37, "grad")


@pytest.mark.parametrize("T,E,K,S,pad,score,z,dtype", [
    (1, 4, 1, 1, 0, "softmax", 0.0, "f32"), (1, 1, 1, 1, 0, "sigmoid", 1e-3, "bf16"),
    (24, 64, 4, 2, 0, "softmax", 1e-3, "f32"), (300, 128, 8, 5, 11, "sigmoid", 0.0, "f32"),
    (257, 130, 3, 3, 0, "softmax", 1e-3, "bf16"), (257, 131, 3, 4, 1, "sigmoid", 1e-3, "bf16"),
    (600, 256, 8, 64, 40, "softmax", 0.0, "bf16"), (90, 512, 22, 1, 0, "sigmoid", 1e-3, "f32"),
    (131, 700, 6, 2, 9, "softmax", 1e-3, "f32"), (131, 701, 6, 131, 0, "sigmoid", 0.0, "f32"),
    (77, 1030, 7, 3, 0, "softmax", 1e-3, "bf16"), (50, 1537, 7, 3, 0, "softmax", 1e-3, "f32"),
    (70, 2047, 36, 2, 3, "sigmoid", 1e-3, "f32"), (64, 2304, 36, 4, 0, "softmax", 1e-3, "f32"),
    (64, 2304, 36, 4, 2, "sigmoid", 0.0, "bf16"), (2500, 64, 6, 7, 100, "softmax", 1e-3, "f32"),
])
def test_balance(R, T, E, K, S, pad, score, z, dtype):
    check_balance(R, T, E, K, sequences(T, S, pad, T + E), score, z, dtype, T + 3 * E)


def test_balance_of_many_short_sequences(R):
    check_balance(R, 2000, 40, 2, sequences(2000, 1000, 30, 3), "softmax", 1e-3, "f32", 4)
    check_balance(R, 600, 2304, 3, sequences(600, 300, 0, 4), "sigmoid", 0.0, "f32", 5)


@pytest.mark.parametrize("T,E,K,seq", [(600_001, 4, 2, None), (3_000_000, 1, 1, (0, 2_999_990)),
                                       (500_000, 60, 2, (5, 250_001, 499_999))])
def test_balance_of_long_batches(R, T, E, K, seq):
    """Sums over up to millions of tokens, against the definition in 64 bits: no team adds up more
    than 256 rows in fp32 (and 32 such sums as one block), what is behind is in 64 bits."""
    gen = torch.Generator(device=DEV).manual_seed(E)
    x = torch.randn(T, E, generator=gen, device=DEV)
    idx = torch.randint(0, E, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    sd = None if seq is None else torch.tensor(seq, dtype=torch.int32, device=DEV)
    loss, counts, _ = R.router_balance_loss_fwd(x, idx, "softmax", 1.0, 0.5, sd)
    ends = (0, T) if seq is None else seq
    want, z = 0.0, 0.0
    for s, (a, b) in enumerate(zip(ends, ends[1:])):
        lse = x[a:b].double().logsumexp(1, keepdim=True)
        c = torch.bincount(idx[a:b].reshape(-1).long(), minlength=E)
        assert torch.equal(c.int(), counts[s])
        want += float(((x[a:b].double() - lse).exp().sum(0) * c).sum()) * E / (K * (b - a) ** 2)
        z += float(lse.square().sum())
    got = loss.double().tolist()
    # a score's own error (softmax of values within 6 of the largest) is random: far below
    # its bound of 50 half steps in such a sum; the additions' as well
    assert abs(got[0] - want / (len(ends) - 1)) <= 64 * STEP * want
    assert abs(got[1] - 0.5 * z / (ends[-1] - ends[0])) <= 512 * STEP * 0.5 * z / (ends[-1] - ends[0]) + 1e-9


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_without_offsets_dropped_choices_wide_logits(R, score):
    check_balance(R, 333, 96, 5, None, score, 1e-3, "f32", 5, scale=8.0, drop=0.3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_balance_at_odd_addresses(R, dtype):
    check_balance(R, 65, 256, 4, sequences(65, 3, 5, 1), "softmax", 1e-3, dtype, 6, off=1)
    check_balance(R, 65, 256, 4, sequences(65, 3, 5, 2), "softmax", 1e-3, dtype, 7, off=2)


def test_balance_padding_in_front_empty_and_one_token_sequences(R):
    seq = np.array([3, 3, 4, 4, 5, 40, 40, 41], np.int32)
    check_balance(R, 50, 72, 3, seq, "softmax", 1e-3, "f32", 8)
    check_balance(R, 50, 72, 3, np.array([50, 50], np.int32), "sigmoid", 1e-3, "f32", 9)
    check_balance(R, 50, 72, 3, np.array([-5, 20, 900], np.int32), "softmax", 0.0, "f32", 10)


def test_balance_of_offsets_out_of_order_stays_within_its_tensors(R):
    # unspecified results, but the tensors around them are left alone
    T, E, K = 64, 40, 2
    pool = torch.full((3, T, E), 5.0, device=DEV)
    x, idx = up(normals((T, E), 1, "f32")), up(choices(T, E, K, 2))
    for order in ([60, 10, 30, 5], [2 ** 31 - 1, -2 ** 31, 7, 7], [0, 64, 0, 64]):
        sd = torch.tensor(order, dtype=torch.int32, device=DEV)
        _, counts, stats = R.router_balance_loss_fwd(x, idx, "softmax", 1.0, 0.1, sd)
        R.router_balance_loss_bwd(torch.ones(2, device=DEV), x, counts, stats, K, "softmax", 1.0,
                                  0.1, sd, grad_logits=pool[1])
        torch.cuda.synchronize()
        assert R.device_status() == 0
        assert bool((pool[0] == 5).all()) and bool((pool[2] == 5).all())


def test_balance_of_no_tokens(R):
    x = torch.empty(0, 32, device=DEV)
    idx = torch.empty(0, 4, dtype=torch.int32, device=DEV)
    for seq in (None, torch.zeros(2, dtype=torch.int32, device=DEV)):
        loss, counts, stats = R.router_balance_loss_fwd(x, idx, "softmax", 1.0, 1.0, seq)
        grad = R.router_balance_loss_bwd(torch.ones(2, device=DEV), x, counts, stats, 4, "softmax",
                                         1.0, 1.0, seq)
        torch.cuda.synchronize()
        assert loss.tolist() == [0.0, 0.0] and int(counts.abs().sum()) == 0
        assert grad.shape == (0, 32) and counts.shape == (1, 32)


def test_balance_is_the_aux_loss_of_one_sequence(R):
    T, E, K = 700, 256, 8
    x = up(normals((T, E), 3, "f32"))
    for score in ("softmax", "sigmoid"):
        q, amap, _ = R.router_aux_scores_fwd(x, K, score)
        aux, tokens = R.router_aux_loss_fwd(q, amap, K, 0.01)
        _, idx, *_ = R.router_topk_fwd_compact(x, K, score)
        loss, counts, _ = R.router_balance_loss_fwd(x, idx, score, 0.01)
        torch.cuda.synchronize()
        assert torch.equal(counts[0], tokens)
        # both within 1e-6 of the exact loss (positive terms; score errors of 2^-21 at most)
        assert abs(float(loss[0]) - float(aux[0])) <= 2e-6 * float(aux[0])


def test_balance_takes_column_views_and_repeats_its_bits(R):
    T, E, K = 1000, 300, 6
    x = up(normals((T, E), 4, "f32"))
    wide = torch.zeros(T, 10, dtype=torch.int32, device=DEV)
    wide[:, 2:8] = up(choices(T, E, K, 5))
    seq = up(sequences(T, 9, 13, 6))
    first = None
    for view in (wide[:, 2:8], wide[:, 2:8].contiguous(), wide[:, 2:8]):
        loss, counts, stats = R.router_balance_loss_fwd(x, view, "sigmoid", 1.0, 0.5, seq)
        grad = R.router_balance_loss_bwd(torch.ones(2, device=DEV), x, counts, stats, K, "sigmoid",
                                         1.0, 0.5, seq)
        inside = stats[:T - 13]
        got = [t.clone() for t in (loss, counts, inside, grad)]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


# ---- quantisation --------------------------------------------------------------------
def check_quantize(R, x, dtype, off=0, q_off=0):
    xd = up(x, dtype)
    if off:
        xd = shifted(xd, off)
    q = torch.empty(x.size + q_off, dtype=torch.int8, device=DEV)[q_off:].view(x.shape)
    q, s = R.router_quantize_rows(xd, out=q)
    torch.cuda.synchronize()
    ref_q, ref_s = B.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref_q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R_,D", [(1, 1), (3, 7), (5, 16), (33, 96), (17, 250), (9, 1001), (70, 2048),
                                  (6, 4104), (3, 8192), (2, 16392), (2, 40000), (2, 65536),
                                  (1, 65535)])
def test_quantize(R, R_, D, dtype):
    check_quantize(R, normals((R_, D), R_ + D, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_ties(R, dtype):
    # every half between two integers, exactly and a step beside it
    rng = np.random.default_rng(3)
    half = (np.arange(-127, 127) + 0.5).astype(np.float32)
    rows = []
    for scale in (1.0, 0.25, 3.0, 1.0 / 3.0, 0.7, 1.9921875):
        top = np.float32(127 * scale)
        if dtype == "bf16":
            top = np.float32(O.round_to_bf16(np.array([top]))[0])
        s = np.float32(np.float64(top) / 127)
        v = (half * s).astype(np.float32)
        for near in (v, np.nextafter(v, np.float32(1e9)), np.nextafter(v, np.float32(-1e9)), top * half / 127):
            row = np.concatenate([near.astype(np.float32), [top], [top / 2, -top / 2]])
            rows.append(row)
    x = np.stack(rows).astype(np.float32)
    if dtype == "bf16":
        x = np.asarray(O.round_to_bf16(x), np.float32)
    check_quantize(R, x, dtype)
    big = (rng.integers(-254, 255, (64, 1000)) / 2.0).astype(np.float32)
    big[:, 0] = 127.0
    check_quantize(R, big if dtype == "f32" else np.asarray(O.round_to_bf16(big), np.float32), dtype)


def test_quantize_large_small_and_empty_rows(R):
    x = normals((8, 64), 5, "f32")
    x[0] = 0.0
    x[1] *= 1e37
    x[2] *= 1e-37
    x[3] *= 1e-40
    x[4] = 0.0
    x[4, 5] = 1.4e-45
    x[5] = -0.0
    x[6, 3] = 3.4e38
    check_quantize(R, x, "f32")
    assert R.router_quantize_rows(torch.empty(0, 8, device=DEV))[0].shape == (0, 8)


def test_quantize_keeps_infinities_and_nan_in_the_scale(R):
    x = normals((4, 300), 6, "f32")
    x[1, 7], x[2, 299], x[3, 0], x[3, 1] = np.inf, np.nan, -np.inf, np.nan
    q, s = R.router_quantize_rows(up(x))
    s, q = s.cpu().numpy(), q.cpu().numpy()
    assert np.isfinite(s[0]) and np.isinf(s[1]) and np.isnan(s[2]) and np.isnan(s[3])
    assert not q[1:].any() and q[0].any()


@pytest.mark.parametrize("dtype,off,q_off", [("f32", 1, 0), ("bf16", 1, 0), ("bf16", 2, 0),
                                             ("bf16", 0, 4), ("f32", 0, 1), ("bf16", 0, 1)])
def test_quantize_at_odd_addresses(R, dtype, off, q_off):
    check_quantize(R, normals((9, 512), 7, dtype), dtype, off, q_off)


# ---- 8-bit products --------------------------------------------------------------------
def int8s(shape, seed, low=-128):
    return np.random.default_rng(seed).integers(low, 128, shape).astype(np.int8)


def w8_tolerance(ref, mag, D, out):
    """Exact products; a fp32 output adds segments of 256 terms or more, each rounded with
    its two scales (three half steps) and added (one each); a bf16 output is one sum,
    exact below 2^24 (up to 1024 terms always) and above that off by at most a step of the
    running sum for each 16 terms."""
    if out == "f32":
        return (3 + D // 256 + 1) * STEP * mag
    s = 4 * STEP * np.abs(ref) + ((D / 16) * 2 * STEP * mag if D > 1024 else 0.0)
    return s + HALF_STEP[out] * (np.abs(ref) + s)


def check_w8(R, m, T, E, K, N, D, out, gather, seed=1, off=0):
    P = T * K
    placed = int(m["off"][-1])
    rows = T if gather else P
    x, w = int8s((rows, D), seed), int8s((E, N, D), seed + 1)
    rng = np.random.default_rng(seed + 2)
    xs = rng.uniform(0.5, 2.0, rows).astype(np.float32)
    ws = rng.uniform(0.001, 0.01, (E, N)).astype(np.float32)
    p2u = m["p2u"] if gather else None
    xd, wd = up(x), up(w)
    if off:
        xd, wd = shifted(xd, off), shifted(wd, off)
    y = torch.full((P, N), 77.0, dtype=DT[out], device=DEV)
    R.router_expert_matmul_w8(xd, up(xs), wd, up(ws), up(m["off"]), up(p2u), out=y,
                              out_dtype=DT[out])
    torch.cuda.synchronize()
    assert R.device_status() == 0
    ref, mag = B.expert_matmul_w8(x, xs, w, ws, m["off"], p2u, T)
    assert_within(down(y)[:placed], ref[:placed], w8_tolerance(ref, mag, D, out)[:placed], "out")
    assert (down(y)[placed:] == 77.0).all()


# one value, one row, whole and ragged tiles, odd rows, many experts, few rows each, pairs
W8 = [
    (1, 1, 1, 1, 1, "f32", True), (1, 4, 1, 8, 16, "bf16", True), (1, 64, 4, 256, 1024, "bf16", True),
    (1, 8, 2, 300, 4112, "f32", True), (3, 5, 5, 33, 17, "bf16", True), (9, 6, 2, 40, 48, "f32", False),
    (32, 64, 8, 128, 512, "bf16", True), (64, 8, 2, 128, 64, "bf16", False),
    (37, 7, 3, 200, 136, "f32", True), (37, 7, 3, 136, 200, "bf16", False),
    (40, 6, 2, 64, 65, "f32", True), (301, 3, 2, 264, 72, "f32", True),
    (129, 16, 4, 320, 336, "bf16", False), (700, 2, 1, 520, 1008, "bf16", True),
    (1100, 1, 1, 136, 272, "f32", True), (515, 4, 2, 257, 255, "bf16", True),
    (515, 4, 2, 257, 260, "f32", True), (70, 300, 6, 24, 40, "f32", True),
    (50, 2304, 36, 16, 32, "bf16", True), (300, 2, 2, 130, 2000, "f32", True),
    (300, 2, 2, 130, 2000, "bf16", False), (600, 3, 1, 384, 1984, "f32", True),
    # several tiles to a CTA and more than one use of every stage, pairs and single CTAs
    (6000, 4, 2, 600, 704, "f32", True), (3000, 40, 3, 1100, 388, "bf16", False),
    (2000, 256, 5, 530, 1040, "bf16", True), (1500, 100, 12, 700, 120, "f32", True),
    # few rows: several tasks to a block, rows in two parts
    (640, 80, 1, 520, 4128, "f32", True), (600, 400, 5, 250, 48, "bf16", True),
]


@pytest.mark.parametrize("T,E,K,N,D,out,gather", W8)
def test_w8(R, T, E, K, N, D, out, gather):
    check_w8(R, route(T, E, K, T + E), T, E, K, N, D, out, gather, seed=N + D)


def test_w8_dropped_choices_and_empty_experts(R):
    for T, K in ((4, 2), (200, 3)):
        m = route(T, 9, K, 3, drop=0.4, empty=(0, 4, 8))
        check_w8(R, m, T, 9, K, 72, 96, "bf16", True)
        check_w8(R, m, T, 9, K, 72, 96, "f32", False)
        m = route(T, 9, K, 4, drop=1.0)
        check_w8(R, m, T, 9, K, 72, 96, "f32", True)


@pytest.mark.parametrize("off", [1, 4, 8])
def test_w8_at_odd_addresses(R, off):
    check_w8(R, route(40, 5, 2, 1), 40, 5, 2, 100, 128, "f32", True, off=off)
    check_w8(R, route(300, 2, 1, 1), 300, 2, 1, 260, 128, "bf16", True, off=off)


@pytest.mark.parametrize("T,E,D", [(400, 2, 960), (400, 2, 4000), (16, 8, 4096), (16, 64, 4096),
                                   (2, 2, 65536)])
def test_w8_exact_integers_of_extreme_operands(R, T, E, D):
    # all products 2^14 or -127 * 128: sums of up to 2^30; fp32 segments add up without error
    # while the running sum stays below 2^24, and within a step of it for each segment above
    N = 130
    m = route(T, E, 1, 2)
    x = np.full((T, D), -128, np.int8)
    w = np.full((E, N, D), -128, np.int8)
    w[:, 1::2] = 127
    ones = np.ones(T, np.float32)
    y = R.router_expert_matmul_w8(up(x), up(ones), up(w), up(np.ones((E, N), np.float32)),
                                  up(m["off"]), up(m["p2u"]), out_dtype=torch.float32)
    got = down(y)
    ref, mag = B.expert_matmul_w8(x, ones, w, np.ones((E, N)), m["off"], m["p2u"], T)
    if D <= 1020:
        assert np.array_equal(got, ref)
    else:
        assert_within(got, ref, (D // 256 + 1) * STEP * mag, "out")


def test_w8_scales_that_are_not_finite_stay_in_their_rows(R):
    T, E, N, D = 40, 4, 64, 64
    for many in (1, 20):
        m = route(T * many, E, 1, 1)
        x, w = int8s((T * many, D), 1), int8s((E, N, D), 2)
        xs = np.ones(T * many, np.float32)
        xs[5], xs[7] = np.nan, np.inf
        y = down(R.router_expert_matmul_w8(up(x), up(xs), up(w), up(np.ones((E, N), np.float32)),
                                           up(m["off"]), up(m["p2u"]), out_dtype=torch.float32))
        token = m["p2u"] % (T * many)
        bad = ~np.isfinite(y).all(axis=1)
        assert set(token[bad]) == {5, 7}


# ---- norms ---------------------------------------------------------------------------------
def make_norm(T, K, D, dtype, gate, post, pre, seed, mapped=True, drop=0.0, E=None):
    m = route(T, E or max(K, 4), K, seed, drop=drop)
    c = {"K": K if mapped else 1, "scale": 0.5, "u2p": m["u2p"] if mapped else None,
         "w": m["w"] if mapped else None,
         "z": normals((T * K if mapped else T, D), seed + 1, dtype),
         "res": normals((T, D), seed + 2, dtype, 2.0),
         "gate": {"none": None, "token": np.abs(normals((T,), seed + 3, "f32")),
                  "value": normals((T, D), seed + 3, dtype)}[gate],
         "post": 1 + 0.2 * normals((D,), seed + 4, "f32") if post else None,
         "pre": 1 + 0.2 * normals((D,), seed + 5, "f32") if pre else None}
    return c


def gate_up(c, dtype):
    return up(c["gate"], dtype if c["gate"] is not None and c["gate"].ndim == 2 else None)


def check_norm(R, c, dtype, off=0):
    z, res = up(c["z"], dtype), up(c["res"], dtype)
    if off:
        z, res = shifted(z, off), shifted(res, off)
    gate = gate_up(c, dtype)
    x, normed, y, rstd = R.router_combine_norm_fwd(
        z, res, up(c["u2p"]), up(c["w"]), post_weight=up(c["post"]), gate=gate,
        residual_scale=c["scale"], pre_weight=up(c["pre"]), eps=1e-5, save=True)
    short = R.router_combine_norm_fwd(
        z, res, up(c["u2p"]), up(c["w"]), post_weight=up(c["post"]), gate=gate,
        residual_scale=c["scale"], pre_weight=up(c["pre"]), eps=1e-5)
    torch.cuda.synchronize()
    assert torch.equal(short[0], x) and short[2] is None and short[3] is None
    ref = B.combine_norm_fwd(c["z"], c["res"], c["u2p"], c["w"], c["post"], c["gate"], c["scale"],
                             c["pre"], np.float64(np.float32(1e-5)))
    tol = norm_tolerances(ref, c, dtype)
    assert_within(down(x), ref["x"], tol["x"], "x")
    assert_within(down(y), ref["y"], tol["y"], "y")
    assert_within(down(rstd), ref["rstd"], tol["rstd"], "rstd")
    if c["pre"] is not None:
        assert torch.equal(short[1], normed)
        assert_within(down(normed), ref["normed"], tol["normed"], "normed")
    else:
        assert normed is None
    # ---- gradients, of what the forward kept
    T, D = c["res"].shape
    gs, gn = normals((T, D), 91, dtype), normals((T, D), 92, dtype)
    gsd, gnd = up(gs, dtype), up(gn, dtype)
    if off:
        gsd = shifted(gsd, off)
    for with_sum in (True, False):
        if not with_sum and c["pre"] is None:
            continue
        got = R.router_combine_norm_bwd(
            gsd if with_sum else None, gnd if c["pre"] is not None else None, y, x, rstd,
            post_weight=up(c["post"]), gate=gate, residual_scale=c["scale"],
            pre_weight=up(c["pre"]))
        torch.cuda.synchronize()
        want = B.combine_norm_bwd(gs if with_sum else None, gn, down(y), down(x), down(rstd),
                                  c["post"], c["gate"], c["scale"], c["pre"])
        names = ("grad_block", "grad_residual", "grad_gate", "grad_post_weight", "grad_pre_weight")
        assert {n for n, t in zip(names, got) if t is not None} == set(want)
        for n, t in zip(names, got):
            if t is not None:
                r, mag = want[n]
                value = c["gate"] is not None and c["gate"].ndim == 2
                assert_within(down(t), r, norm_grad_tolerance(n, r, mag, T, dtype, value), n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "token", "value"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_norm_forms(R, dtype, gate, post, pre):
    check_norm(R, make_norm(37, 3, 264, dtype, gate, post, pre, 11), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,D", [(1, 1, 1), (1, 8, 2048), (5, 36, 40), (3, 33, 2), (1000, 2, 24),
                                   (700, 4, 257), (130, 2, 1026), (33, 2, 4096), (19, 3, 4100),
                                   (21, 1, 5001), (11, 2, 8192), (9, 2, 8191)])
def test_norm_sizes(R, T, K, D, dtype):
    check_norm(R, make_norm(T, K, D, dtype, "token" if D % 2 else "value", True, True, T + D), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_without_a_map_dropped_choices_odd_addresses(R, dtype):
    check_norm(R, make_norm(50, 1, 512, dtype, "none", True, True, 1, mapped=False), dtype)
    check_norm(R, make_norm(50, 4, 512, dtype, "token", True, True, 2, drop=0.5), dtype)
    check_norm(R, make_norm(50, 2, 512, dtype, "token", True, True, 3, drop=1.0), dtype)
    check_norm(R, make_norm(50, 2, 512, dtype, "value", True, True, 4), dtype, off=1)
    check_norm(R, make_norm(50, 2, 512, dtype, "value", True, True, 5), dtype, off=2)


def test_norm_is_the_combination_bit_for_bit(R):
    c = make_norm(64, 8, 2048, "bf16", "none", True, True, 6)
    z, u2p, w = up(c["z"], "bf16"), up(c["u2p"]), up(c["w"])
    *_, y, _ = R.router_combine_norm_fwd(z, up(c["res"], "bf16"), u2p, w, post_weight=up(c["post"]),
                                         save=True)
    assert torch.equal(y, R.router_combine_fwd(z, u2p, 8, w))


def test_norm_of_no_rows(R):
    e = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    x, n, y, r = R.router_combine_norm_fwd(e, e, post_weight=w, pre_weight=w, save=True)
    assert x.shape == n.shape == y.shape == (0, 64) and r.shape == (0, 2)
    *_, gate, gpost, gpre = R.router_combine_norm_bwd(e, e, y, x, r, post_weight=w, pre_weight=w)
    torch.cuda.synchronize()
    assert gate is None and not gpost.any() and not gpre.any()


def test_norm_backward_against_differences(R):
    """The forward's own outputs along a direction (fp32, a sum over all outputs): central
    differences of a step of 2^-6 are off by its square and the forward's rounding over it."""
    T, K, D = 6, 2, 96
    c = make_norm(T, K, D, "f32", "value", True, True, 12)
    c["w"][:] = 1.0
    gs, gn = normals((T, D), 1, "f32"), normals((T, D), 2, "f32")

    def value(**change):
        d = {**c, **change}
        x, n, y, r = R.router_combine_norm_fwd(
            up(d["z"]), up(d["res"]), up(d["u2p"]), up(d["w"]), post_weight=up(d["post"]),
            gate=up(d["gate"]), residual_scale=0.5, pre_weight=up(d["pre"]), save=True)
        return float((down(x) * gs).sum() + (down(n) * gn).sum()), (x, y, r)

    _, (x, y, r) = value()
    gb, gr, gg, gpost, gpre = R.router_combine_norm_bwd(
        up(gs), up(gn), y, x, r, post_weight=up(c["post"]), gate=up(c["gate"]), residual_scale=0.5,
        pre_weight=up(c["pre"]))
    gz, _ = R.router_combine_bwd(gb, up(c["u2p"]), K, None, up(c["w"]))
    step = 2.0 ** -6
    for name, grad in (("z", gz), ("res", gr), ("gate", gg), ("post", gpost), ("pre", gpre)):
        d = normals(c[name].shape, 77, "f32")
        up_, down_ = (value(**{name: (c[name] + s * step * d).astype(np.float32)})[0] for s in (1, -1))
        want = float((down(grad) * d).sum())
        size = float(np.linalg.norm(down(grad)) * np.linalg.norm(d))
        assert abs((up_ - down_) / (2 * step) - want) <= 2e-3 * size, name


# ---- together -----------------------------------------------------------------------------------
def block(R, s, stream=None):
    """An expert block for serving on 8-bit weights, and its training losses."""
    x, normed, _, _ = R.router_combine_norm_fwd(s["y0"], s["res"], post_weight=s["wpost"],
                                                pre_weight=s["wpre"])
    logits = normed.float() @ s["wr"]
    w, idx, _, off, p2u, u2p, _ = R.router_topk_fwd_maps(logits, s["K"], "softmax_post",
                                                         workspace=s.get("maps_ws"))
    q, qs = R.router_quantize_rows(normed)
    h = R.router_expert_matmul_w8(q, qs, s["w1"], s["s1"], off, p2u)
    a = torch.relu(h)
    q2, q2s = R.router_quantize_rows(a)
    z = R.router_expert_matmul_w8(q2, q2s, s["w2"], s["s2"], off)
    out = R.router_combine_norm_fwd(z, x, u2p, w, post_weight=s["wpost"], gate=s["gate"],
                                    residual_scale=0.5, pre_weight=s["wpre"], save=True)
    loss, counts, stats = R.router_balance_loss_fwd(logits, idx, "softmax", 0.01, 1e-3, s["seq"])
    grad = R.router_balance_loss_bwd(s["ones"], logits, counts, stats, s["K"], "softmax", 0.01,
                                     1e-3, s["seq"])
    grads = R.router_combine_norm_bwd(s["g"], s["g"], out[2], out[0], out[3],
                                      post_weight=s["wpost"], gate=s["gate"], residual_scale=0.5,
                                      pre_weight=s["wpre"])
    return dict(x=x, normed=normed, logits=logits, w=w, idx=idx, off=off, p2u=p2u, u2p=u2p, q=q, qs=qs,
                h=h, q2=q2, q2s=q2s, z=z, sum=out[0], normed2=out[1], y=out[2], rstd=out[3],
                loss=loss, counts=counts, grad=grad, gb=grads[0], gr=grads[1], gg=grads[2],
                gpost=grads[3], gpre=grads[4])


def block_state(T, E, K, D, N, seed):
    rng = np.random.default_rng(seed)
    return {"K": K, "y0": up(normals((T, D), seed, "bf16"), "bf16"),
            "res": up(normals((T, D), seed + 1, "bf16"), "bf16"),
            "wpost": up(1 + 0.1 * normals((D,), seed + 2, "f32")),
            "wpre": up(1 + 0.1 * normals((D,), seed + 3, "f32")),
            "wr": up(normals((D, E), seed + 4, "f32", D ** -0.5)),
            "w1": up(int8s((E, N, D), seed + 5)), "w2": up(int8s((E, D, N), seed + 6)),
            "s1": up(rng.uniform(1e-4, 1e-3, (E, N)).astype(np.float32)),
            "s2": up(rng.uniform(1e-4, 1e-3, (E, D)).astype(np.float32)),
            "gate": up(rng.uniform(0, 1, T).astype(np.float32)),
            "seq": up(sequences(T, 3, T // 8, seed)), "ones": torch.ones(2, device=DEV),
            "g": up(normals((T, D), seed + 7, "bf16"), "bf16")}


@pytest.mark.parametrize("T,E,K,D,N", [(4, 32, 4, 256, 128), (300, 16, 4, 256, 160),
                                       (1500, 8, 2, 128, 272)])
def test_block_together(R, T, E, K, D, N):
    s = block_state(T, E, K, D, N, T)
    r = block(R, s)
    torch.cuda.synchronize()
    assert R.device_status() == 0
    host = {k: down(v) for k, v in r.items()}
    off, p2u, u2p = (r[k].cpu().numpy() for k in ("off", "p2u", "u2p"))
    # each step on what the one before gave
    ref, scales = B.quantize_rows(host["normed"])
    assert np.array_equal(r["q"].cpu().numpy(), ref) and np.array_equal(r["qs"].cpu().numpy(), scales)
    for name, (q, qs, w, ws, p) in {"h": ("q", "qs", "w1", "s1", p2u),
                                    "z": ("q2", "q2s", "w2", "s2", None)}.items():
        want, mag = B.expert_matmul_w8(host[q], host[qs], down(s[w]), down(s[ws]), off, p, T)
        assert_within(host[name], want, w8_tolerance(want, mag, s[w].shape[2], "bf16"), name)
    ref, scales = B.quantize_rows(np.maximum(host["h"], 0.0))
    assert np.array_equal(r["q2"].cpu().numpy(), ref) and np.array_equal(r["q2s"].cpu().numpy(), scales)
    c = {"K": K, "scale": 0.5, "gate": down(s["gate"]), "post": down(s["wpost"]),
         "pre": down(s["wpre"])}
    want = B.combine_norm_fwd(host["z"], host["x"], u2p, host["w"], c["post"], c["gate"], 0.5,
                              c["pre"], np.float64(np.float32(1e-6)))
    tol = norm_tolerances(want, c, "bf16")
    for name, key in (("sum", "x"), ("normed2", "normed"), ("y", "y"), ("rstd", "rstd")):
        assert_within(host[name], want[key], tol[key], name)
    want, counts = B.balance_loss(host["logits"], r["idx"].cpu().numpy(), "softmax",
                                  np.float64(np.float32(0.01)), np.float64(np.float32(1e-3)),
                                  s["seq"].cpu().numpy())
    assert np.array_equal(r["counts"].cpu().numpy(), counts)
    assert_within(host["loss"], want, balance_loss_tolerance(host["logits"], "softmax", want), "loss")


def test_block_in_a_graph_and_on_streams(R):
    s, other = block_state(200, 16, 4, 256, 160, 1), block_state(200, 16, 4, 256, 160, 2)
    for st in (s, other):
        st["maps_ws"] = torch.empty(
            R.lib().router_expert_maps_workspace_bytes(200, 16), dtype=torch.uint8, device=DEV)
    want, want_other = block(R, s), block(R, other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(R, s)
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        held_other = block(R, other)
    side = torch.cuda.Stream()
    for _ in range(3):
        for t in list(held.values()) + list(held_other.values()):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()  # the two graphs at once, each with its own workspaces
        with torch.cuda.stream(side):
            second.replay()
            loose = block(R, other)
        torch.cuda.synchronize()
        inside = {"stats"}
        for k in want:
            if k in inside:
                continue
            assert torch.equal(held[k], want[k]), k
            assert torch.equal(held_other[k], want_other[k]), k
            assert torch.equal(loose[k], want_other[k]), k
    # new inputs in the captured tensors
    for k in ("y0", "res", "gate", "seq"):
        s[k].copy_(other[k])
    for k in ("wpost", "wpre", "wr", "w1", "w2", "s1", "s2", "g"):
        s[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    for k in want_other:
        assert torch.equal(held[k], want_other[k]), k


def test_refusals_on_the_gpu(R):
    x = torch.zeros(4, 32, dtype=torch.int8, device=DEV)
    w = torch.zeros(2, 8, 32, dtype=torch.int8, device=DEV)
    one, off = torch.ones(4, device=DEV), torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    ws = torch.ones(2, 8, device=DEV)
    for bad in (dict(x=x.float()), dict(w=w[:, :, ::2]), dict(xs=one[:3]), dict(xs=one.double()),
                dict(ws=ws[:1]), dict(off=off[:2]), dict(out_dtype=torch.float16),
                dict(w=w.cpu()), dict(x=x[:, :16])):
        a = dict(x=x, xs=one, w=w, ws=ws, off=off, out_dtype=None) | bad
        with pytest.raises(ValueError):
            R.router_expert_matmul_w8(a["x"], a["xs"], a["w"], a["ws"], a["off"],
                                      out_dtype=a["out_dtype"])
    rows = torch.zeros(4, 32, device=DEV)
    v = torch.ones(32, device=DEV)
    for bad in (dict(gate=one.bfloat16()), dict(gate=rows[:, :3]), dict(post_weight=v[:5]),
                dict(pre_weight=v.double()), dict(z=rows[:3]), dict(z=rows.bfloat16()),
                dict(topk_weights=rows[:, :1]), dict(normed=rows.clone())):
        a = dict(z=rows) | bad
        with pytest.raises(ValueError):
            R.router_combine_norm_fwd(a.pop("z"), rows, **a)
    with pytest.raises(R.RouterError):
        R.router_combine_norm_fwd(rows, rows, eps=0.0)
    with pytest.raises(R.RouterError):
        big = torch.zeros(1, 8200, device=DEV)
        R.router_combine_norm_fwd(big, big)
    for args in ((None, None, rows, rows, None), (None, rows, rows, rows, None),
                 (rows, None, rows, rows, torch.ones(4, 2, device=DEV))):
        with pytest.raises(ValueError):
            R.router_combine_norm_bwd(*args, post_weight=v, pre_weight=v if args[0] is not None else None)
    idx = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    for bad in (dict(idx=idx.long()), dict(idx=idx[:3]), dict(seq=off.long()), dict(seq=off[:1]),
                dict(score="softmax_post"), dict(seq=torch.zeros(6, dtype=torch.int32, device=DEV))):
        a = dict(idx=idx, seq=None, score="softmax") | bad
        with pytest.raises((ValueError, R.RouterError)):
            R.router_balance_loss_fwd(rows, a["idx"], a["score"], 1.0, 0.0, a["seq"])
    with pytest.raises(R.RouterError):
        R.router_balance_loss_fwd(rows, idx, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
