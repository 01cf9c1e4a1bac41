"""The operators around the routed experts where batches, scales and logits are unusual,
against the definitions in 64 bits."""
import numpy as np
import pytest

from blocks_cases import HALF_STEP, STEP, normals, score_error

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


# ---- balance loss -------------------------------------------------------------------
def exact_balance(x, idx, g, score, coeff, z, seq):
    """(loss [2], counts, stats, grad, mag of grad) of sequences seq, in 64 bits; stats and
    grad of padding are zeros."""
    T, E = x.shape
    K, S = idx.shape[1], len(seq) - 1
    x = x.double()
    n = max(seq[-1] - seq[0], 1)
    loss = torch.zeros(2, dtype=torch.float64, device=DEV)
    counts = torch.zeros(S, E, dtype=torch.int32, device=DEV)
    stats = torch.zeros(T, 2, dtype=torch.float64, device=DEV)
    grad, mag = torch.zeros_like(x), torch.zeros_like(x)
    for s, (a, b) in enumerate(zip(seq, seq[1:])):
        if a == b:
            continue
        r = x[a:b]
        top = r.amax(1, keepdim=True)
        total = (r - top).exp().sum(1, keepdim=True)
        lse = top + total.log()
        soft, sig = (r - top).exp() / total, torch.sigmoid(r)
        norm = sig.sum(1, keepdim=True)
        q = soft if score == "softmax" else sig / norm
        w = soft if score == "softmax" else sig * torch.sigmoid(-r) / norm
        stats[a:b] = torch.cat((top, total) if score == "softmax" else (norm, lse), 1)
        chosen = idx[a:b].reshape(-1).long()
        c = torch.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        counts[s] = c.int()
        c = c.double()
        by = coeff * E / (S * K * (b - a) ** 2)
        loss[0] += by * (q.sum(0) * c).sum()
        loss[1] += z / n * lse.square().sum()
        dz = g[1] * z * 2 / n * lse * soft
        grad[a:b] = g[0] * by * w * (c - (q * c).sum(1, keepdim=True)) + dz
        c = (c - (b - a) * K / E).abs()  # a constant less changes nothing
        mag[a:b] = abs(g[0] * by) * w * (c + (q * c).sum(1, keepdim=True)) + dz.abs()
    return loss, counts, stats, grad, mag


def within(got, want, tol, name):
    off = (got.double() - want).abs() - tol
    assert not bool(torch.isnan(got).any()), name
    assert float(off.max()) <= 0.0, (name, float(off.max()))


def errors(x, score):
    """score_error of the logits, and of the softmax, without those whose score is zero in any
    arithmetic (and minus infinity)."""
    x = x.double()
    top = x.amax(1, keepdim=True)
    x = torch.where(x < top - 200.0, top, x).cpu().numpy()
    return score_error(x, score), score_error(x, "softmax")


def check_rows(x, idx, score, z, seq, out, dtype, g):
    """Each row's kept numbers and gradient, and the counts."""
    _, counts, stats, grad = out
    _, want_counts, want_stats, want, mag = exact_balance(x, idx, g, score, 0.01, z, seq)
    assert torch.equal(counts, want_counts)
    error, soft_error = errors(x, score)
    inside = slice(seq[0], seq[-1])
    if score == "softmax":
        assert torch.equal(stats[inside, 0].double(), want_stats[inside, 0])  # the maximum
    else:
        within(stats[inside, 0], want_stats[inside, 0], error * want_stats[inside, 0], "stats")
    if score == "softmax":
        within(stats[inside, 1], want_stats[inside, 1], error * want_stats[inside, 1], "stats")
    tol = (2 * error + soft_error + 48 * STEP) * mag  # as for rows without padding
    within(grad, want, tol + HALF_STEP[dtype] * (want.abs() + tol) + 1e-37, "grad")


# Padding in front of the first sequence, more rows to a team than it has under way (3 at 2304
# experts, 4 or 8 at 512): the rows behind it are not computed from those of the padding.
@pytest.mark.parametrize("T,E,K,front,score,z,dtype", [
    (65536, 512, 22, 100, "softmax", 1e-3, "f32"), (65536, 512, 22, 5003, "sigmoid", 0.0, "f32"),
    (65536, 512, 22, 131, "softmax", 1e-3, "bf16"), (65536, 512, 22, 9999, "sigmoid", 1e-3, "bf16"),
    (8192, 2304, 36, 101, "softmax", 1e-3, "f32"), (8192, 2304, 36, 3005, "sigmoid", 1e-3, "bf16"),
    (30000, 64, 4, 70, "softmax", 0.0, "f32"), (30000, 66, 4, 70, "softmax", 1e-3, "f32"),
])
def test_balance_of_left_padded_batches(R, T, E, K, front, score, z, dtype):
    gen = torch.Generator(device=DEV).manual_seed(T + E + front)
    x = torch.randn(T, E, generator=gen, device=DEV).to(DT[dtype])
    idx = torch.randint(0, E, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    seq = [front, front, front + 1, (front + T) // 2, T - 7, T - 7]
    sd = torch.tensor(seq, dtype=torch.int32, device=DEV)
    g = [0.75, 1.25]
    first = None
    for other in (0.0, 30.0, -5.0):  # what the padding's rows hold changes no bit
        x[:front] = other + torch.randn(front, E, generator=gen, device=DEV).to(DT[dtype])
        idx[:front] = torch.randint(0, E, (front, K), generator=gen, device=DEV, dtype=torch.int32)
        loss, counts, stats = R.router_balance_loss_fwd(x, idx, score, 0.01, z, sd)
        grad = torch.full((T, E), 77.0, dtype=DT[dtype], device=DEV)
        R.router_balance_loss_bwd(torch.tensor(g, device=DEV), x, counts, stats, K, score, 0.01, z,
                                  sd, grad_logits=grad)
        got = [loss, counts, stats[front:T - 7], grad]
        if first is None:
            first = got
            check_rows(x, idx, score, z, seq, (loss, counts, stats, grad), dtype, g)
        assert all(torch.equal(a, b) for a, b in zip(first, got))
        assert not bool(grad[:front].any()) and not bool(grad[T - 7:].any())


# Masked experts: the type's lowest value, minus infinity, or far below the others.  At 2304 experts a
# row is two warps': with all but 128 neighbouring experts masked one of them has none left.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score,z", [("softmax", 1e-3), ("softmax", 0.0), ("sigmoid", 1e-3),
                                     ("sigmoid", 0.0)])
@pytest.mark.parametrize("E,left", [(2304, range(128, 256)), (2304, range(0, 100)),
                                    (2303, range(1300, 1400)), (512, range(7, 9)), (96, range(95, 96))])
def test_balance_of_masked_experts(R, E, left, score, z, dtype):
    T, K = 150, min(4, len(left))
    x = up(normals((T, E), E, "f32"))
    gen = torch.Generator(device=DEV).manual_seed(E)
    idx = left[0] + torch.randint(0, len(left), (T, K), generator=gen, device=DEV, dtype=torch.int32)
    off = torch.ones(E, dtype=torch.bool, device=DEV)
    off[left[0]:left[-1] + 1] = False
    for mask in (torch.finfo(DT[dtype]).min, -float("inf"), -1e4):
        x[:, off] = mask
        xd = x.to(DT[dtype])
        loss, counts, stats = R.router_balance_loss_fwd(xd, idx, score, 0.01, z)
        g = [0.75, 1.25]
        grad = R.router_balance_loss_bwd(torch.tensor(g, device=DEV), xd, counts, stats, K, score,
                                         0.01, z)
        check_rows(xd, idx, score, z, [0, T], (loss, counts, stats, grad), dtype, g)
        want = exact_balance(xd, idx, g, score, 0.01, z, [0, T])[0]
        error, soft = errors(xd, score)
        # 150 tokens are added up one behind the other at most; the z loss takes two errors of lse,
        # which is below 10 and, as a mean of squares here, above 0.1
        assert float((loss[0] - want[0]).abs()) <= (error + 150 * STEP) * float(want[0])
        assert float((loss[1] - want[1]).abs()) <= (20 * soft + 160 * STEP) * float(want[1]) + 1e-37


@pytest.mark.parametrize("E", [64, 1000, 2304])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_balance_of_rows_at_the_ends_of_the_type(R, dtype, E):
    """Rows with every expert masked by the lowest value, or with logits next to the largest: the
    softmax of equal logits, or of one above all others."""
    T, K = 24, 2
    x = up(normals((T, E), E, "f32"))
    ends = torch.finfo(DT[dtype])
    x[1] = ends.min
    x[2] = ends.max
    x[3] = ends.min
    x[3, E - 1] = ends.max
    x[4] = 2.0 ** 120
    x[4, 5] = 2.0 ** 121
    x[5] = -2.0 ** 99
    x[6] = -2.0 ** 100
    x[6, 0] = -2.0 ** 101
    xd = x.to(DT[dtype])
    idx = torch.arange(T * K, device=DEV, dtype=torch.int32).view(T, K) % E
    loss, counts, stats = R.router_balance_loss_fwd(xd, idx, "softmax", 0.01)
    grad = R.router_balance_loss_bwd(torch.ones(2, device=DEV), xd, counts, stats, K, "softmax", 0.01)
    check_rows(xd, idx, "softmax", 0.0, [0, T], (loss, counts, stats, grad), dtype, [1.0, 1.0])
    want = exact_balance(xd, idx, [1.0, 1.0], "softmax", 0.01, 0.0, [0, T])[0]
    assert float((loss[0] - want[0]).abs()) <= (errors(xd, "softmax")[0] + 64 * STEP) * float(want[0])


def test_balance_gradient_of_counts_above_2_to_the_24(R):
    """Two experts that are chosen nearly alike by 40 million tokens: the gradient is of the
    difference of two counts that fp32 does not hold."""
    T, E = 40_000_000, 2
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.rand(T, E, generator=gen, device=DEV)
    idx = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    idx[:T // 2 - 501] = 1
    _, counts, stats = R.router_balance_loss_fwd(x, idx, "softmax", 1.0)
    assert counts.tolist() == [[T // 2 + 501, T // 2 - 501]]
    grad = R.router_balance_loss_bwd(torch.tensor([1e12, 0.0], device=DEV), x, counts, stats, 1, "softmax", 1.0)
    error = score_error(np.array([[0.0, 1.0]]), "softmax")  # logits within one of each other
    for a in range(0, T, 8_000_000):
        q = x[a:a + 8_000_000].double().softmax(1)
        c = torch.tensor([501.0, -501.0], dtype=torch.float64, device=DEV)  # less their mean
        by = 1e12 * E / T ** 2
        inner = (q * c).sum(1, keepdim=True)
        mag = by * q * (c.abs() + (q * c.abs()).sum(1, keepdim=True))
        within(grad[a:a + 8_000_000], by * q * (c - inner), (3 * error + 48 * STEP) * mag, "grad")


# ---- 8-bit products --------------------------------------------------------------------
# up to eight rows an expert, 30 and 350: the kernel of few rows, single CTAs and pairs
@pytest.mark.parametrize("T,E", [(3, 2), (40, 8), (640, 80), (60, 2), (700, 2)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_w8_of_very_small_and_very_large_rows(R, T, E, out):
    """Scales whose product is subnormal or infinite where the output is a number."""
    from blocks_cases import B, route
    N, D = 72, 128
    m = route(T, E, 1, T)
    rng = np.random.default_rng(T)
    x, w = rng.integers(-128, 128, (T, D)).astype(np.int8), rng.integers(-128, 128, (E, N, D)).astype(np.int8)
    xs = rng.uniform(0.5, 1.0, T).astype(np.float32)
    ws = rng.uniform(0.5, 1.0, (E, N)).astype(np.float32)
    xs[0], xs[1], xs[2] = 2.0 ** -126, 8e-37, 8e35
    xs[3:] *= np.float32(2.0) ** rng.integers(-100, 100, T - 3).astype(np.float32)
    ws[:, ::3] *= np.float32(1e-6)
    ws[:, 1::3] *= np.float32(1e3)
    w[:, 1] = 0  # sums of zero stay zero beside scales of 8e35 and 1e3
    y = R.router_expert_matmul_w8(up(x), up(xs), up(w), up(ws), up(m["off"]), up(m["p2u"]), out_dtype=DT[out])
    got = y.double().cpu().numpy()
    ref, mag = B.expert_matmul_w8(x, xs, w, ws, m["off"], m["p2u"], T)
    # the sums are exact (below 2^24): two products, each rounded to 2^-24 of itself or (the second
    # one) half the smallest number
    tol = 2 * STEP * np.abs(ref) + 2.0 ** -150
    if out == "bf16":
        tol = tol + HALF_STEP[out] * (np.abs(ref) + tol) + 2.0 ** -134
    large = np.abs(ref) > 3.38e38  # infinite, or next to it
    assert np.isinf(got[np.abs(ref) > 3.5e38]).all() and large.any() and not large.all()
    assert (np.abs(got - ref) <= tol)[~large].all()
    assert not got[:, 1].any()


@pytest.mark.parametrize("T,E,N,D", [(6000, 2, 600, 960), (3000, 40, 1100, 384), (4096, 4, 512, 128)])
def test_w8_of_many_tiles_to_a_pair_is_exact(R, T, E, N, D):
    """Every integer of many stages that pass between the CTAs of a pair, on data that change from
    call to call: sums below 2^24 are exact, and a second call gives the same."""
    per = T // E
    off = torch.arange(E + 1, device=DEV, dtype=torch.int32) * per
    gen = torch.Generator(device=DEV).manual_seed(D)
    for _ in range(6):
        x = torch.randint(-128, 128, (T, D), generator=gen, device=DEV, dtype=torch.int8)
        w = torch.randint(-128, 128, (E, N, D), generator=gen, device=DEV, dtype=torch.int8)
        one, ones = torch.ones(T, device=DEV), torch.ones(E, N, device=DEV)
        y = R.router_expert_matmul_w8(x, one, w, ones, off, out_dtype=torch.float32)
        want = torch.bmm(x.view(E, per, D).double(), w.double().transpose(1, 2)).view(T, N)
        assert torch.equal(y.double(), want)
        assert torch.equal(y, R.router_expert_matmul_w8(x, one, w, ones, off, out_dtype=torch.float32))
    assert R.device_status() == 0


# One sequence of nearly all tokens among short ones, in front, behind and between them: the
# second kernel's warps add its slots up together.  (E 66: rows that are not aligned.)
@pytest.mark.parametrize("T,E,K,S,place,dtype", [
    (65536, 64, 6, 64, 0, "f32"), (65536, 64, 6, 64, 63, "bf16"), (65536, 66, 6, 80, 40, "f32"),
    (8192, 2304, 4, 64, 5, "f32"), (30000, 130, 3, 700, 699, "f32"), (30000, 128, 3, 700, 350, "f32"),
])
def test_balance_of_one_long_sequence_among_short_ones(R, T, E, K, S, place, dtype):
    gen = torch.Generator(device=DEV).manual_seed(T + S)
    x = torch.randn(T, E, generator=gen, device=DEV).to(DT[dtype])
    idx = torch.randint(0, E, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    short = 5
    seq = [i * short for i in range(place + 1)] + [T - (S - 1 - i) * short for i in range(place, S)]
    sd = torch.tensor(seq, dtype=torch.int32, device=DEV)
    g = [0.75, 1.25]
    loss, counts, stats = R.router_balance_loss_fwd(x, idx, "softmax", 0.01, 1e-3, sd)
    grad = R.router_balance_loss_bwd(torch.tensor(g, device=DEV), x, counts, stats, K, "softmax", 0.01,
                                     1e-3, sd)
    check_rows(x, idx, "softmax", 1e-3, seq, (loss, counts, stats, grad), dtype, g)
    want = exact_balance(x, idx, g, "softmax", 0.01, 1e-3, seq)[0]
    # at most 256 rows behind one another in a team's sums, and some 50 additions behind those
    error, soft = errors(x, "softmax")
    assert float((loss[0] - want[0]).abs()) <= (error + 306 * STEP) * float(want[0])
    assert float((loss[1] - want[1]).abs()) <= (soft + 320 * STEP) * float(want[1])
    again = R.router_balance_loss_fwd(x, idx, "softmax", 0.01, 1e-3, sd)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts)


# Up to eight rows an expert on average with some experts of many: two kernels share the experts.
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("sizes,N,D", [
    ((32, 33, 0, 1, 600, 31, 0, 129, 2, 128), 1024, 1008), ((1200,), 1030, 1024), ((), 2048, 512),
    ((33,) * 40, 1000, 1024), ((300, 128, 127, 500), 600, 4096)])
def test_w8_of_a_few_hot_experts(R, sizes, N, D, gather):
    E = 320
    rng = np.random.default_rng(len(sizes) + N)
    n = rng.integers(0, 8, E)
    n[rng.permutation(E)[:len(sizes)]] = sizes
    P, owned = 2400, int(n.sum())
    assert owned <= P <= 8 * E and P * N * D > 2 ** 31
    off = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(N)
    T = 300 if gather else P
    x = torch.randint(-127, 128, (T, D), generator=gen, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (E, N, D), generator=gen, device=DEV, dtype=torch.int8)
    p2u = torch.randperm(P, generator=gen, device=DEV).int() if gather else None
    one, ones = torch.ones(T, device=DEV), torch.ones(E, N, device=DEV)
    y = torch.full((P, N), 0.5, device=DEV)
    R.router_expert_matmul_w8(x, one, w, ones, off, p2u, out=y, out_dtype=torch.float32)
    rows = x[p2u.long() % T] if gather else x
    cut = off.tolist()
    for e in range(E):
        a, b = cut[e], cut[e + 1]
        want = rows[a:b].double() @ w[e].double().t()
        if D <= 1024:  # sums below 2^24
            assert torch.equal(y[a:b].double(), want), e
        elif b > a:  # parts of at least 256 terms, added up in round-to-nearest
            mag = rows[a:b].double().abs() @ w[e].double().abs().t()
            within(y[a:b], want, (D // 256 + 1) * STEP * mag, e)
    assert bool((y[owned:] == 0.5).all())
    again = R.router_expert_matmul_w8(x, one, w, ones, off, p2u, out=torch.full_like(y, 0.5),
                                      out_dtype=torch.float32)
    assert torch.equal(y, again) and R.device_status() == 0


# ---- norms ---------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,gate", [(24, "none"), (257, "token"), (2048, "value"), (4100, "token")])
def test_norms_keep_nan_and_infinities_in_their_rows(R, D, gate, dtype):
    """Forward and backward: the rows without one get the same bits as beside ordinary rows."""
    T = 61
    bad = {3: float("nan"), 17: float("inf"), 60: -float("inf")}
    ok = torch.ones(T, dtype=torch.bool, device=DEV)
    ok[list(bad)] = False
    clean = {k: up(normals((T, D), 10 + i, dtype), dtype) for i, k in enumerate(("z", "res", "gs", "gn"))}
    wpost, wpre = up(1 + 0.1 * normals((D,), 1, "f32")), up(1 + 0.1 * normals((D,), 2, "f32"))
    g = {"none": None, "token": up(np.abs(normals((T,), 3, "f32"))),
         "value": up(normals((T, D), 3, dtype), dtype)}[gate]

    def run(t):
        x, n, y, r = R.router_combine_norm_fwd(t["z"], t["res"], post_weight=wpost, gate=g,
                                               residual_scale=0.5, pre_weight=wpre, save=True)
        gb, gr, gg, _, _ = R.router_combine_norm_bwd(t["gs"], t["gn"], y, x, r, post_weight=wpost, gate=g,
                                                     residual_scale=0.5, pre_weight=wpre)
        return [v for v in (x, n, y, r, gb, gr, gg) if v is not None]

    want = run(clean)
    for name in clean:
        dirty = dict(clean)
        dirty[name] = clean[name].clone()
        for row, value in bad.items():
            dirty[name][row, (row * 7) % D] = value
        got = run(dirty)
        for a, b in zip(want, got):
            assert torch.equal(a[ok], b[ok]), name
        # and where they are they show: x for the forward's inputs, the residual's gradient behind
        shown = got[0] if name in ("z", "res") else got[5]
        assert not bool(torch.isfinite(shown[~ok]).all(1).any()), name


# ---- captured -------------------------------------------------------------------------------
def test_replays_follow_the_offsets(R):
    """What the kernels decide on the device (hot experts, a long sequence, padding in front) is
    decided again by each replay: a graph captured on even batches, two replays under way at once."""
    E, P, N, D, T, S, K = 320, 2400, 1024, 1008, 20000, 64, 4
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randint(-127, 128, (P, D), generator=gen, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (E, N, D), generator=gen, device=DEV, dtype=torch.int8)
    xs = torch.rand(P, generator=gen, device=DEV)
    ws = torch.rand(E, N, generator=gen, device=DEV)
    logits = torch.randn(T, 64, generator=gen, device=DEV)
    idx = torch.randint(0, 64, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    hot = np.full(E, 2)
    hot[[7, 200]] = 1100, 400
    offsets = [np.concatenate([[0], np.cumsum(n)]).clip(max=P) for n in (np.full(E, 7), hot, np.eye(E)[9] * P)]
    seqs = [np.arange(S + 1) * (T // S), np.concatenate([[500], 600 + 5 * np.arange(S - 1), [T - 3]]),
            np.concatenate([[0], T - 5 * np.arange(S - 1, -1, -1)])]
    states = [(up(offsets[0]).int(), up(seqs[0]).int()) for _ in range(2)]
    one = torch.ones(2, device=DEV)

    def call(off, seq):
        y = R.router_expert_matmul_w8(x, xs, w, ws, off)
        loss, counts, stats = R.router_balance_loss_fwd(logits, idx, "softmax", 0.01, 1e-3, seq)
        return y, loss, counts, R.router_balance_loss_bwd(one, logits, counts, stats, K, "softmax", 0.01,
                                                          1e-3, seq)

    call(*states[0])
    graphs, held = [], []
    for state in states:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(call(*state))
    side = torch.cuda.Stream()
    for a, b in ((0, 1), (1, 2), (2, 0)):
        want = []
        for (off, seq), i in zip(states, (a, b)):
            off.copy_(up(offsets[i]))
            seq.copy_(up(seqs[i]))
            want.append(call(off, seq))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for got, exp, i in zip(held, want, (a, b)):
            owned = int(offsets[i][-1])
            assert torch.equal(got[0][:owned], exp[0][:owned])
            assert all(torch.equal(p, q) for p, q in zip(got[1:], exp[1:]))
    assert R.device_status() == 0
