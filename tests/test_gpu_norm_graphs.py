"""GPU tests of the norm and its gradient of more rows than one launch takes: two streams at once, and a captured step that is
replayed with other inputs."""
import pytest
import torch

from gpu_util import log

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


@pytest.mark.parametrize("n,dim", [(2100, 1160), (5000, 136), (1030, 20008), (1025, 65536)])
def test_streams_and_graph(wc, n, dim):
    def draw(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return [torch.randn(n, dim, generator=g, device="cuda").to(BF16) for _ in range(3)]

    x, r, dy = draw(9)
    w = torch.rand(dim, device="cuda").to(BF16)
    need = wc.rms_norm_grad_work_bytes(n, dim)

    def state():
        return dict(sum=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(n, device="cuda"),
                    dh=torch.empty_like(x), dw=torch.empty(dim, device="cuda"),
                    work=torch.empty(need, dtype=torch.uint8, device="cuda"))

    def step(s, stream=None):
        wc.rms_norm_async(x, w, n, dim, 1e-5, y_dev=s["y"], residual_dev=r, sum_dev=s["sum"], rstd_dev=s["rstd"],
                          stream=stream)
        wc.rms_norm_grad_async(dy, s["sum"], w, s["rstd"], n, dim, s["dh"], s["dw"], s["work"], need, dsum_dev=s["y"],
                               stream=stream)

    def same(a, b):
        return all(torch.equal(a[k], b[k]) for k in ("sum", "y", "rstd", "dh", "dw"))

    log(f"case: rms_norm and its gradient, {n}x{dim}, on two streams and captured")
    want, a, b = state(), state(), state()
    step(want)
    torch.cuda.synchronize()
    step(a, torch.cuda.Stream())
    step(b, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert same(a, want) and same(b, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for seed in range(3):
        for t, new in zip((x, r, dy), draw(seed)):
            t.copy_(new)
        step(want)
        graph.replay()
        torch.cuda.synchronize()
        assert same(a, want)
