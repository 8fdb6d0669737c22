"""GPU tests of products with matrices of e4m3 codes that have scales per block of 128."""
import pytest
import torch

from e4m3_ref import BLOCK, UBF16, _largest_of_eights, blocks, gemm_tolerance, matrix_codes, per_column, quantised, values_of, within
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn
GUARD = 64


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _case(rows, cols, tokens, seed):
    """(codes, scales, the matrix; codes, scales, the activations), the matrices they stand for in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g).float())
    codes, scales, w = matrix_codes(w)
    x = torch.randn(tokens, cols, generator=g) * torch.exp2(torch.randint(-6, 7, (tokens, 1), generator=g).float())
    x[:, ::61] *= 20
    xc, xs = quantised(x)
    return codes, scales, w, xc, xs, values_of(xc) * per_column(xs, cols)


def _run(wc, W, xc, xs, tokens, out, **kw):
    n = tokens * W.rows
    y = torch.full((n + GUARD,), -7.0, dtype=BF16 if out == "bf16" else torch.float32, device="cuda")
    need = wc.gemm_fp8_work_bytes(W, tokens)
    work = torch.full((need + GUARD,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN wherever it is read unwritten
    wc.gemm_fp8_async(W, xc, xs, tokens, y, work if need else None, need, out=out, **kw)
    torch.cuda.synchronize()
    assert bool((y[n:] == -7.0).all()) and bool((work[need:] == 0xFF).all()), "wrote past the end"
    return y[:n].reshape(tokens, W.rows)


SHAPES = [(1, 16, 1), (3, 32, 2), (16, 128, 1), (17, 144, 3), (128, 128, 16), (129, 256, 17), (100, 1168, 5),
          (1000, 512, 1), (1024, 4096, 1), (64, 28672, 2), (333, 2096, 40), (1003, 2096, 65), (256, 1024, 128),
          (257, 640, 129), (515, 384, 300), (2000, 272, 33), (4096, 128, 9), (96, 65536, 3), (1, 4096, 500),
          (2, 144, 1025), (640, 1536, 700), (1027, 1040, 515), (5000, 256, 2), (9000, 400, 24)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,tokens", SHAPES)
def test_products(wc, rows, cols, tokens, out):
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, rows + cols + tokens)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens, {out}")
    W = wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols)
    y = _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)
    want = x @ w.t()
    assert within(y, want, gemm_tolerance(x, w, out == "bf16", want))
    again = _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)
    assert torch.equal(y, again), "two runs differ"


# tiles of every size, whole and cut at rows, tokens and columns; sums in one part and in up to 16
TILES = [(1304, 2704, 90), (1003, 2096, 333), (1027, 1040, 515), (1001, 4112, 1000), (5000, 1008, 200), (1000, 2064, 1200),
         (1601, 800, 2000), (4100, 656, 1030), (4352, 128, 4100), (8200, 400, 2049), (4100, 656, 4352), (4097, 272, 4097),
         (64, 28672, 40), (97, 65536, 70), (300, 20000, 64), (130, 16400, 300), (1024, 14336, 100), (2050, 8208, 130),
         (4096, 14336, 128), (8192, 4112, 16), (8209, 4112, 31), (9001, 1296, 5)]


# a matrix that one tile of tokens reads once, whose tiles and groups begin at different blocks of columns; groups of 16, 32
# and 64 rows on either side of where they are taken
ONCE = [(12000, 144, 60), (16400, 272, 100), (28672, 272, 60), (28673, 400, 64), (9000, 2064, 50), (14337, 400, 509),
        (4096, 400, 3), (4097, 1168, 16), (10239, 272, 16), (10240, 400, 5), (10241, 1296, 16), (16384, 272, 1), (16385, 272, 16),
        (10250, 400, 32), (4100, 272, 17)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,tokens", TILES + ONCE)
def test_tiles(wc, rows, cols, tokens, out):
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, rows)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens, {out}")
    W = wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols)
    y = _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)
    xd, wd = x.cuda(), w.cuda()
    want = xd @ wd.t()
    tol = 2.0 ** -23 * (128 + 2 * blocks(cols) + 4) * (xd.abs() @ wd.abs().t()) + 1e-40
    if out == "bf16":
        tol += 2.0 ** -11 * _largest_of_eights(x, w).cuda()
        tol += UBF16 * (want.abs() + tol)
    assert within(y, want.cpu(), tol.cpu())
    again = _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)
    assert torch.equal(y, again), "two runs differ"


@pytest.mark.parametrize("tokens", list(range(1, 20)) + [31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128])
def test_few_tokens(wc, tokens):
    rows, cols = 272, 1296
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, tokens)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens")
    y = _run(wc, wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols), xc.cuda(), xs.cuda(), tokens, "f32")
    want = x @ w.t()
    assert within(y, want, gemm_tolerance(x, w, False, want))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 24, 200])
def test_every_code(wc, tokens, out):
    """Each of the 254 finite codes times each other: single products, of 8 bits, are exact in fp32 and in bf16."""
    cols, rows = 128, 254
    finite = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    codes = torch.zeros(rows, cols, dtype=torch.uint8)
    codes[:, 77] = finite
    log(f"case: gemm_fp8 every code, {tokens} tokens")
    W = wc.Fp8Matrix(codes.cuda(), torch.ones(2, 1, device="cuda"), rows, cols)
    for start in range(0, 254, tokens):
        mine = finite[start:start + tokens]
        xc = torch.zeros(len(mine), cols, dtype=torch.uint8)
        xc[:, 77] = mine
        y = _run(wc, W, xc.cuda(), torch.ones(len(mine), 1, device="cuda"), len(mine), out)
        assert torch.equal(y.cpu().double(), values_of(mine)[:, None] * values_of(finite)[None, :])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 20, 150])
def test_columns_of_blocks(wc, tokens, out):
    """Every column reaches the right block's scales: one nonzero column at a time, scales all different."""
    rows, cols = 300, 400
    g = torch.Generator().manual_seed(1)
    scales = torch.exp2(torch.randint(-8, 8, (3, 4), generator=g).float())
    xs = torch.exp2(torch.randint(-8, 8, (tokens, 4), generator=g).float())
    log(f"case: gemm_fp8 columns one by one, {tokens} tokens")
    for c in (0, 15, 16, 63, 64, 127, 128, 255, 256, 383, 384, 399):
        codes, xc = torch.zeros(rows, cols, dtype=torch.uint8), torch.zeros(tokens, cols, dtype=torch.uint8)
        codes[:, c] = torch.randint(1, 127, (rows,), generator=g).to(torch.uint8)
        xc[:, c] = torch.randint(1, 127, (tokens,), generator=g).to(torch.uint8)
        W = wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols)
        y = _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)
        want = (values_of(xc[:, c]) * xs.double()[:, c // BLOCK])[:, None] * \
            (values_of(codes[:, c]) * scales.double()[torch.arange(rows) // BLOCK, c // BLOCK])[None]
        assert torch.equal(y.cpu().double(), want), c


@pytest.mark.parametrize("rows,cols,tokens", [(256, 512, 1), (256, 512, 20), (300, 400, 200)])
def test_no_numbers_stay_among_themselves(wc, rows, cols, tokens):
    """A NaN code or scale reaches its own row or token alone, also where tiles reach past the ends."""
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, 9)
    log(f"case: gemm_fp8 NaN, {rows}x{cols}, {tokens} tokens")
    want = x @ w.t()
    tol = gemm_tolerance(x, w, False, want)
    bad = codes.view(torch.uint8).clone()
    bad[rows - 1, cols - 1] = 0x7F
    y = _run(wc, wc.Fp8Matrix(bad.cuda(), scales.cuda(), rows, cols), xc.cuda(), xs.cuda(), tokens, "f32")
    assert bool(torch.isnan(y[:, rows - 1]).all()) and within(y[:, :rows - 1], want[:, :-1], tol[:, :-1])
    xs[tokens - 1, 0] = float("nan")
    y = _run(wc, wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols), xc.cuda(), xs.cuda(), tokens, "f32")
    assert bool(torch.isnan(y[tokens - 1]).all())
    if tokens > 1:
        assert within(y[:-1], want[:-1], tol[:-1])


def test_views_streams_and_graph(wc):
    """Operands that lie inside larger tensors whose neighbours are NaN codes, two streams at once, and captured calls
    that are replayed with other activations."""
    rows, cols = 520, 1296
    big = torch.full((rows * cols + 512,), 0x7F, dtype=torch.uint8, device="cuda")
    for tokens in (1, 7, 150):
        codes, scales, w, xc, xs, x = _case(rows, cols, tokens, tokens + 3)
        log(f"case: gemm_fp8 views, streams and graph, {tokens} tokens")
        view = big[256:256 + rows * cols]
        view.copy_(codes.view(torch.uint8).flatten())
        wide = torch.full((tokens * cols + 512,), 0x7F, dtype=torch.uint8, device="cuda")
        mine = wide[256:256 + tokens * cols]
        mine.copy_(xc.view(torch.uint8).flatten())
        xsd = torch.full((tokens * blocks(cols) + 64,), float("nan"), device="cuda")[32:-32]
        xsd.copy_(xs.flatten())
        W = wc.Fp8Matrix(view, scales.cuda(), rows, cols)
        want = x @ w.t()
        y = _run(wc, W, mine, xsd, tokens, "f32")
        assert within(y, want, gemm_tolerance(x, w, False, want))
        need = wc.gemm_fp8_work_bytes(W, tokens)
        calls = [(torch.cuda.Stream(), torch.empty(tokens, rows, device="cuda"),
                  torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")) for _ in range(2)]
        torch.cuda.synchronize()
        for stream, out, work in calls:
            wc.gemm_fp8_async(W, mine, xsd, tokens, out, work, need, out="f32", stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(out, y) for _, out, _ in calls)
        out, work = calls[0][1:]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            wc.gemm_fp8_async(W, mine, xsd, tokens, out, work, need, out="f32")
        for seed in range(3):
            other, others = quantised(torch.randn(tokens, cols, generator=torch.Generator().manual_seed(seed)))
            mine.copy_(other.view(torch.uint8).flatten())
            xsd.copy_(others.flatten())
            eager = _run(wc, W, mine, xsd, tokens, "f32")
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager)


def test_nothing(wc):
    e = torch.empty(0, device="cuda")
    W = wc.Fp8Matrix(torch.zeros(32, 64, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda"), 32, 64)
    assert wc.gemm_fp8_work_bytes(W, 0) == 0
    wc.gemm_fp8_async(W, e.to(torch.uint8), e, 0, e.to(BF16), None, 0)
    none = wc.Fp8Matrix(e.to(torch.uint8), e, 0, 64)
    wc.gemm_fp8_async(none, torch.zeros(5, 64, dtype=torch.uint8, device="cuda"), torch.ones(5, 1, device="cuda"), 5, e,
                      None, 0, out="f32")


@pytest.mark.parametrize("tokens", [1, 40])
def test_large_scales(wc, tokens):
    """Scales far from one whose product is in range."""
    rows, cols = 130, 384
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, 4)
    log(f"case: gemm_fp8 large and small scales, {tokens} tokens")
    W = wc.Fp8Matrix(codes.cuda(), (scales * 2.0 ** 90).cuda(), rows, cols)
    y = _run(wc, W, xc.cuda(), (xs * 2.0 ** -90).cuda(), tokens, "f32")
    want = x @ w.t()
    assert within(y, want, gemm_tolerance(x, w, False, want))


@pytest.mark.parametrize("tokens", [1, 20, 60, 300])
def test_sums_that_cancel(wc, tokens):
    """Large products that cancel beside small ones: fp32 results, and those of few tokens, keep the small ones whole."""
    rows, cols = 200, 256
    codes, xc = torch.zeros(rows, cols), torch.zeros(tokens, cols)
    codes[:, 0], codes[:, 1], xc[:, 0], xc[:, 1] = 448.0, -448.0, 448.0, 448.0
    codes[:, 2:], xc[:, 2:] = 0.125, 0.0625                   # 254 products of 2^-7, beside 448 * 448
    xc[:, 128:130] = 0.0625
    log(f"case: gemm_fp8 cancelling sums, {tokens} tokens")
    W = wc.Fp8Matrix(codes.to(F8).cuda(), torch.ones(2, 2, device="cuda"), rows, cols)
    y = _run(wc, W, xc.to(F8).cuda(), torch.ones(tokens, 2, device="cuda"), tokens, "f32")
    # in any order each partial sum is a multiple of 2^-7 below 2^18: up to one bit more than fp32 holds is lost per sum
    assert bool(((y.cpu().double() - 254 / 128).abs() <= 128 * 2.0 ** -7).all())
    alone = torch.zeros(tokens, cols)
    alone[:, 2:] = xc[:, 2:]
    y = _run(wc, W, alone.to(F8).cuda(), torch.ones(tokens, 2, device="cuda"), tokens, "f32")
    assert torch.equal(y.cpu().double(), torch.full((tokens, rows), 254 / 128, dtype=torch.float64))
