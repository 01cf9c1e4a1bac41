"""How far the expert products' fp32 outputs are from 64 bits, as a whole: relative
2-norm errors, which see a loss of precision that element-wise bounds (the sum of
the terms' magnitudes times their number) leave room for.

The bound.  A tensor core adds 16 products to its accumulator by truncation, below
the 24 bits of the sum: a chain of n additions loses at most n steps of 2^-25 of its
value and n 2^-26 on average, all towards zero, so that a segment of n = 60 (960
terms) is off by 60 2^-26 = 9.0e-7 of its value, as is a sum of segments whose signs
differ.  Rounding to nearest at each segment's end, at most 2^-24 of the running sum
and as often up as down, adds 2^-24 sqrt(k / 12) for k segments: 5.2e-8 at 9 of them,
in square 3e-15 beside 8e-13.  Together below 1e-6.  A chain over 2000 terms without
segments would be off by 1.9e-6.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BOUND = 1e-6


@pytest.fixture(scope="module")
def R():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from score_top_expert_gb300 import build
    build.build()
    import score_top_expert_gb300.router as r
    r.lib()
    return r


def inputs(T, E, K, N, D, dtype, gather, seed=3):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normals(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(DT[dtype])

    P = T * K
    expert = torch.randint(0, E, (P,), generator=gen, device=DEV).sort().values
    off = torch.searchsorted(expert, torch.arange(E + 1, device=DEV)).int()
    p2u = torch.randperm(P, generator=gen, device=DEV).int() if gather else None
    x, w, g = normals(T if gather else P, D), normals(E, N, D, scale=D ** -0.5), normals(P, N)
    rows = x if p2u is None else x[(p2u % T).long()]
    return x, w, g, off, p2u, rows.double()


def relative(got, ref):
    assert torch.isfinite(got).all()
    return float((got.double() - ref).norm() / ref.norm())


def by_expert(a, off, m):
    """[P, :] rows of each expert times m(e)."""
    o = off.tolist()
    return torch.cat([a[o[e]:o[e + 1]] @ m(e) for e in range(len(o) - 1)])


# few rows: four warps to a tile (a quarter of the contraction each), and one
@pytest.mark.parametrize("T,E,K,N,D", [
    (6, 4, 4, 264, 520), (6, 4, 4, 264, 2000), (6, 4, 4, 264, 8000), (1, 1, 1, 40, 65536),
    (36, 36, 1, 4096, 512), (36, 36, 1, 4096, 2008), (36, 36, 1, 2304, 8000)])
def test_few_rows(R, T, E, K, N, D):
    x, w, _, off, p2u, rows = inputs(T, E, K, N, D, "bf16", True)
    y = R.router_expert_matmul(x, w, off, p2u, out_dtype=torch.float32)
    ref = by_expert(rows, off, lambda e: w[e].double().t())
    assert relative(y, ref) <= BOUND


# rows an expert: 25 take single CTAs on the tensor cores, 50 and more pairs; widths in
# eights the copy engine, others and fp32 the element loads
@pytest.mark.parametrize("length", [504, 2000, 8000])
@pytest.mark.parametrize("dtype,odd,gather", [("bf16", 0, True), ("bf16", 0, False),
                                              ("bf16", 1, True), ("f32", 0, True),
                                              ("f32", 1, False)])
@pytest.mark.parametrize("rows", [25, 50])
def test_products_over_long_contractions(R, length, dtype, odd, gather, rows):
    E, K = 8, 2
    T, short, long = rows * E // K, 136 + odd, length + odd
    x, w, _, off, p2u, xr = inputs(T, E, K, short, long, dtype, gather)
    y = R.router_expert_matmul(x, w, off, p2u, out_dtype=torch.float32)
    assert relative(y, by_expert(xr, off, lambda e: w[e].double().t())) <= BOUND
    _, w, g, off, _, _ = inputs(T, E, K, long, short, dtype, gather, seed=4)
    gx = R.router_expert_matmul_bwd_input(g, w, off, out_dtype=torch.float32)
    assert relative(gx, by_expert(g.double(), off, lambda e: w[e].double())) <= BOUND


# columns of grad_out: up to 128 single CTAs, more pairs
@pytest.mark.parametrize("length", [500, 2000, 8000])
@pytest.mark.parametrize("dtype,odd,gather", [("bf16", 0, True), ("bf16", 0, False),
                                              ("bf16", 1, True), ("f32", 0, True),
                                              ("f32", 1, False)])
@pytest.mark.parametrize("N", [72, 264])
def test_weight_gradient_over_many_rows(R, length, dtype, odd, gather, N):
    # two experts of about `length` rows
    x, _, g, off, p2u, xr = inputs(length, 2, 2, N + odd, 136 + odd, dtype, gather)
    gw = R.router_expert_matmul_bwd_weight(g, x, off, p2u, out_dtype=torch.float32)
    o = off.tolist()
    ref = torch.stack([g[o[e]:o[e + 1]].double().t() @ xr[o[e]:o[e + 1]] for e in range(2)])
    assert relative(gw, ref) <= BOUND


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T,E,K,N", [(1, 4, 2, 264), (30, 40, 4, 1000)])
def test_w4_over_long_rows(R, group, T, E, K, N):
    D = 8192
    x, _, _, off, p2u, xr = inputs(T, E, K, 8, D, "bf16", True)
    gen = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randint(0, 256, (E, N, D // 2), generator=gen, device=DEV, dtype=torch.uint8)
    s = (torch.rand(E, N, D // group, generator=gen, device=DEV) + 0.5).bfloat16()
    y = R.router_expert_matmul_w4(x, q, s, off, p2u, out_dtype=torch.float32)

    def weight(e):
        w = torch.stack((q[e] & 15, q[e] >> 4), 2).view(N, -1, group).double() - 8
        return (w * s[e].double()[..., None]).view(N, D).t()

    assert relative(y, by_expert(xr, off, weight)) <= BOUND


@pytest.mark.parametrize("exponent", [-100, -112, -120, -128, -136, -146])
def test_tiny_fp32_operands_are_cut_at_2_to_the_minus_133(R, exponent):
    # bf16 parts end at 2^-133: an operand counts as its multiple of that next to zero,
    # so a product is off by at most 2^-133 times the other operand (at least 2^-133),
    # and the sum of those is all that comes to the bound of ordinary operands
    T, E, K, N, D = 40, 4, 2, 72, 130
    x, w, g, off, p2u, _ = inputs(T, E, K, N, D, "f32", True)
    x = (x.double() * 2.0 ** exponent).float()
    w = w * 2.0 ** 100
    y = R.router_expert_matmul(x, w, off, p2u).double()
    xr = x[(p2u % T).long()].double()
    ref = by_expert(xr, off, lambda e: w[e].double().t())
    mag = by_expert(xr.abs(), off, lambda e: w[e].double().abs().t())
    cut = by_expert(torch.ones_like(xr), off, lambda e: w[e].double().abs().t()) * 2.0 ** -133
    assert ((y - ref).abs() <= (D + 2) * 2.0 ** -23 * (mag + cut) + cut).all()
    # bf16 operands have no parts below it
    xb, wb = x.bfloat16(), w.bfloat16()
    y = R.router_expert_matmul(xb, wb, off, p2u, out_dtype=torch.float32).double()
    xr = xb[(p2u % T).long()].double()
    ref = by_expert(xr, off, lambda e: wb[e].double().t())
    mag = by_expert(xr.abs(), off, lambda e: wb[e].double().abs().t())
    assert ((y - ref).abs() <= (D + 2) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("dtype,odd,segment", [("bf16", 0, 960), ("bf16", 1, 960), ("f32", 0, 512)])
def test_tiny_results_of_segmented_sums(R, dtype, odd, segment):
    # adding a segment may leave zero for a result below 2^-126: at most that much for
    # each addition, beside the bound of the sums (and the cut of fp32 operands)
    T, E, K, N, D = 100, 4, 2, 72, 2000 + odd
    x, w, g, off, p2u, _ = inputs(T, E, K, N, D, dtype, True)
    x, w = x * 2.0 ** -66, w * 2.0 ** -62
    y = R.router_expert_matmul(x, w, off, p2u, out_dtype=torch.float32).double()
    xr = x[(p2u % T).long()].double()
    ref = by_expert(xr, off, lambda e: w[e].double().t())
    mag = by_expert(xr.abs(), off, lambda e: w[e].double().abs().t())
    assert ref.abs().max() < 2.0 ** -125
    steps = -(-D // segment)
    assert ((y - ref).abs() <= (D + 2) * (2.0 ** -23 * mag + 2.0 ** -149) + steps * 2.0 ** -126).all()
