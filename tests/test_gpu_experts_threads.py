"""Expert-side calls from several host threads at once, each on a stream and sizes of
its own, through the C entry points (which other threads run beside)."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"


@pytest.fixture(scope="module")
def R():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from score_top_expert_gb300 import build
    build.build()
    import score_top_expert_gb300.router as r
    r.lib()
    return r


def relative(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def test_three_host_threads_with_kernels_of_other_sizes(R):
    L = R.lib()
    P, N = 8, 64
    # one kernel, three sizes of shared memory
    sizes = {"small": (4, 64), "large": (2304, 4096), "between": (600, 2048)}
    start, results = threading.Barrier(len(sizes)), {}

    def calls(name, E, D):
        gen = torch.Generator(device=DEV).manual_seed(D)
        off = torch.full((E + 1,), P, device=DEV, dtype=torch.int32)
        off[0] = 0
        x = torch.randn(P, D, generator=gen, device=DEV).bfloat16()
        w = torch.randn(1, N, D, generator=gen, device=DEV).bfloat16()
        q = torch.randint(0, 256, (E, N, D // 2), generator=gen, device=DEV, dtype=torch.uint8)
        s = torch.rand(E, N, D // 32, generator=gen, device=DEV).bfloat16()
        y4, y = torch.empty(P, N, device=DEV), torch.empty(P, N, device=DEV)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        start.wait()
        codes = set()
        for _ in range(20):
            codes.add(L.router_expert_matmul_w4(
                x.data_ptr(), q.data_ptr(), s.data_ptr(), None, 32, off.data_ptr(), None, P, P, E,
                N, D, y4.data_ptr(), 0, stream.cuda_stream))
            codes.add(L.router_expert_matmul(x.data_ptr(), 1, w.data_ptr(), off.data_ptr(), None,
                                             P, P, 1, N, D, y.data_ptr(), 0, stream.cuda_stream))
        stream.synchronize()
        wide = torch.stack((q[0] & 15, q[0] >> 4), 2).view(N, -1, 32).double() - 8
        wide = (wide * s[0].double()[..., None]).view(N, D)
        results[name] = (codes, relative(y4, x.double() @ wide.t()),
                         relative(y, x.double() @ w[0].double().t()))

    threads = [threading.Thread(target=calls, args=(n, *v)) for n, v in sizes.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert set(results) == set(sizes)
    for name, (codes, w4, product) in results.items():
        # relative 2-norms of fp32 sums, at most 4096 terms in segments of at most 128
        assert codes == {0} and w4 <= 1e-6 and product <= 1e-6, (name, codes, w4, product)
