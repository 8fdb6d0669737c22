"""GPU tests of activations to e4m3 codes with a scale per 128 columns."""
import pytest
import torch

from e4m3_ref import U32, blocks, check_codes, values_of
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
GUARD = 64


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _run(wc, x, n, dim, gated, **kw):
    codes = torch.full((n * dim + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((n * blocks(dim) + GUARD,), -7.0, device="cuda")
    wc.quant_fp8_async(x, n, dim, codes, scales, gated=gated, **kw)
    torch.cuda.synchronize()
    assert bool((codes[n * dim:] == 0x5A).all()) and bool((scales[n * blocks(dim):] == -7.0).all()), "wrote past the end"
    return codes[:n * dim].reshape(n, dim), scales[:n * blocks(dim)].reshape(n, -1)


def _exact(x, dim, gated):
    """(y, how far fp32 may be off it): silu's exponential has a rounded argument (2^-24 |gate| log2(e), taken twice for
    the function's own steps) and is within 2^-22, the sum, the reciprocal (2^-23) and two products follow."""
    y = x.cpu().double()
    if not gated:
        return y, torch.zeros_like(y)
    gate, up = y[:, :dim], y[:, dim:]
    y = gate * torch.sigmoid(gate) * up
    return y, ((3 * gate.abs() + 12) * U32) * y.abs() + 1e-37 * up.abs()


SHAPES = [(1, 8), (3, 16), (1, 128), (2, 136), (5, 1160), (37, 1168), (1, 4096), (64, 4096), (7, 14336), (3, 28680),
          (2, 65536), (1031, 256), (300, 520)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n,dim", SHAPES)
def test_codes(wc, n, dim, gated):
    g = torch.Generator().manual_seed(n + dim)
    x = torch.randn(n, dim * (2 if gated else 1), generator=g)
    x[:, ::97] *= 30
    x = x.to(BF16)
    log(f"case: quant_fp8 {n}x{dim} gated {gated}")
    codes, scales = _run(wc, x.cuda(), n, dim, gated)
    check_codes(codes, scales, *_exact(x, dim, gated))
    again = _run(wc, x.cuda(), n, dim, gated)
    assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])


@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -101, 2.0 ** -60, 2.0 ** 60, 2.0 ** 120])
def test_sizes_of_values(wc, size):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(4, 264, generator=g) * size).to(BF16)
    x[1] = 0
    x[2, 128:] = 0
    log(f"case: quant_fp8 values of {size:g}")
    codes, scales = _run(wc, x.cuda(), 4, 264, False)
    check_codes(codes, scales, *_exact(x, 264, False))
    assert bool((values_of(codes)[1] == 0).all()) and bool(torch.isfinite(scales).all())


def test_every_word(wc):
    """Every finite bf16 word, 128 words of one exponent to a block: the codes are the nearest."""
    words = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(BF16)
    x = torch.stack((words, -words)).reshape(2 * 255, 128)
    log("case: quant_fp8 of every finite word")
    codes, scales = _run(wc, x.cuda(), 510, 128, False)
    check_codes(codes, scales, *_exact(x, 128, False))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_blocks_without_a_number(wc, bad):
    """The block that holds it is NaN, and no other."""
    x = torch.ones(3, 400).to(BF16)
    x[1, 200] = bad
    log(f"case: quant_fp8 {bad}")
    codes, scales = _run(wc, x.cuda(), 3, 400, False)
    want = torch.zeros(3, 4, dtype=torch.bool)
    want[1, 1] = True
    assert torch.equal(torch.isnan(scales).cpu(), want)
    ok = torch.ones(3, 400, dtype=torch.bool)
    ok[1, 128:256] = False
    assert bool((values_of(codes)[ok] == 448).all())


def test_gate_far_from_zero(wc):
    """silu of large gates is the gate, of large negative ones zero, not NaN."""
    gate = torch.tensor([-3e38, -1e4, -200.0, -90.0, -80.0, 0.0, 80.0, 1e4])
    x = torch.cat((gate, torch.full((8,), 2.0)))[None].to(BF16)
    log("case: quant_fp8 gates far from zero")
    codes, scales = _run(wc, x.cuda(), 1, 8, True)
    y = _exact(x, 8, True)
    check_codes(codes, scales, y[0], y[1])


def test_another_stream_and_graph(wc):
    n, dim = 33, 1160
    g = torch.Generator().manual_seed(8)
    x = torch.randn(n, 2 * dim, generator=g).to(BF16).cuda()
    want = _run(wc, x, n, dim, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(wc, x, n, dim, True, stream=side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    codes, scales = torch.empty(n, dim, dtype=F8, device="cuda"), torch.empty(n, blocks(dim), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wc.quant_fp8_async(x, n, dim, codes, scales, gated=True)
    for seed in range(3):
        x.copy_(torch.randn(n, 2 * dim, generator=torch.Generator().manual_seed(seed)))
        want = _run(wc, x, n, dim, True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(codes.view(torch.uint8), want[0]) and torch.equal(scales, want[1])


def test_nothing(wc):
    empty = torch.empty(0, device="cuda")
    wc.quant_fp8_async(empty.to(BF16), 0, 128, empty.to(torch.uint8), empty)
