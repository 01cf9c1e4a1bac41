"""Infinities and NaN among fp32 operands of the expert products: the results that
the definition has in fp32, where a number's parts may be empty."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
INF = float("inf")


@pytest.fixture(scope="module")
def R():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from score_top_expert_gb300 import build
    build.build()
    import score_top_expert_gb300.router as r
    r.lib()
    return r


def numbers(shape, seed, exact):
    """Numbers away from zero; ``exact``: those of bf16 (only a first part)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    a = torch.randn(*shape, generator=gen, device=DEV)
    a = torch.where(a < 0, a - 0.1, a + 0.1)
    return a.bfloat16().float() if exact else a


E, P, N = 3, 60, 72
OFF = [0, 20, 21, 60]


def product(a, w, off):
    """[P, :] rows times their expert's matrix, in 64 bits."""
    return torch.cat([a[off[e]:off[e + 1]].double() @ w[e].double() for e in range(E)])


def same_specials(got, ref):
    """Infinities with their signs and NaN where the definition has them."""
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isposinf(), ref.isposinf())
    assert torch.equal(got.isneginf(), ref.isneginf())


# 64 terms, several slices, several segments
@pytest.mark.parametrize("D", [64, 257, 1301])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_an_infinity_gives_infinities(R, D, exact, out):
    off = torch.tensor(OFF, device=DEV, dtype=torch.int32)
    x, w, g = numbers((P, D), 1, exact), numbers((E, N, D), 2, exact), numbers((P, N), 3, exact)
    x[3, 5], x[3, 60], x[30, D - 1], x[45, 0], x[45, 1] = INF, INF, -INF, INF, -INF
    w[0, 7, 9] = -INF
    g[10, 4], g[59, N - 1] = INF, -INF
    y = R.router_expert_matmul(x, w, off, out_dtype=out)
    ref = product(x, w.transpose(1, 2), OFF)
    assert ref.isinf().sum() > N and ref.isnan().any()
    same_specials(y, ref)
    gx = R.router_expert_matmul_bwd_input(g, w, off, out_dtype=out)
    ref = product(g, w, OFF)
    assert ref.isinf().sum() > D
    same_specials(gx, ref)
    gw = R.router_expert_matmul_bwd_weight(g, x, off, out_dtype=out)
    ref = torch.stack([g[OFF[e]:OFF[e + 1]].double().t() @ x[OFF[e]:OFF[e + 1]].double()
                       for e in range(E)])
    assert ref.isinf().sum() > D
    same_specials(gw, ref)


def test_an_infinity_times_zero_is_a_nan(R):
    off = torch.tensor(OFF, device=DEV, dtype=torch.int32)
    x, w = numbers((P, 64), 1, True), numbers((E, N, 64), 2, True)
    x[3, 5] = INF
    w[0, 7, 5] = 0.0
    y = R.router_expert_matmul(x, w, off)
    same_specials(y, product(x, w.transpose(1, 2), OFF))
    assert y[3].isnan().sum() == 1


@pytest.mark.parametrize("bits", [0x7f800001, 0x7f80ffff, -0x007fffff, 0x7fc00000, 0x7fffffff])
def test_a_nan_of_any_bits_stays_a_nan(R, bits):
    # 0x7f800001: nothing of its fraction is in the upper half
    off = torch.tensor(OFF, device=DEV, dtype=torch.int32)
    w, g = numbers((E, N, 130), 2, False), numbers((P, N), 3, False)

    def with_nan(shape, seed, *at):
        a = numbers(shape, seed, False)
        a.view(torch.int32)[at] = bits
        assert a[at].isnan()
        return a

    x = with_nan((P, 130), 1, 20, 100)
    y = R.router_expert_matmul(x, w, off)
    assert y[20].isnan().all() and y[:20].isfinite().all() and y[21:].isfinite().all()
    gw = R.router_expert_matmul_bwd_weight(g, x, off)
    assert gw[1, :, 100].isnan().all() and gw.isnan().sum() == N
    y = R.router_expert_matmul(numbers((P, 130), 1, False), with_nan((E, N, 130), 2, 2, 5, 64), off)
    assert y[21:, 5].isnan().all() and y.isnan().sum() == P - 21
    gx = R.router_expert_matmul_bwd_input(with_nan((P, N), 3, 59, 1), w, off)
    assert gx[59].isnan().all() and gx[:59].isfinite().all()
