"""Norms, codes, products and clipping where an offset in elements passes 2^31 and 2^32: rows behind it are what a call on
those rows alone gives, or what 64 bits give."""
import pytest
import torch

from e4m3_ref import gemm_tolerance, matrix_codes, per_column, quantised, values_of, within
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
N, DIM = 1 << 20, 4104   # 2^32 + 2^23 elements
ROWS = [0, (1 << 31) // DIM - 1, (1 << 31) // DIM, (1 << 32) // DIM - 1, (1 << 32) // DIM, N - 2, N - 1]


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    yield mod
    torch.cuda.empty_cache()


def _rows(seed):
    x = torch.empty(N, DIM, dtype=BF16, device="cuda")
    piece = torch.randn(1 << 14, DIM, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)
    for k in range(0, N, 1 << 14):
        x[k:k + (1 << 14)] = piece
    x[ROWS] = torch.randn(len(ROWS), DIM, device="cuda").to(BF16)   # no other row is like these
    return x


def test_codes_and_norm(wc):
    blocks = -(-DIM // 128)
    log(f"case: quant_fp8 and rms_norm {N}x{DIM}")
    x, w = _rows(1), torch.rand(DIM, device="cuda").to(BF16)
    codes = torch.empty(N, DIM, dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, blocks, device="cuda")
    some = x[ROWS].clone()
    n = len(ROWS)
    codes1, scales1 = torch.empty(n, DIM, dtype=torch.uint8, device="cuda"), torch.empty(n, blocks, device="cuda")
    wc.quant_fp8_async(x, N, DIM, codes, scales)
    wc.quant_fp8_async(some, n, DIM, codes1, scales1)
    assert torch.equal(codes[ROWS], codes1) and torch.equal(scales[ROWS], scales1)
    total, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(N, device="cuda")
    total1, y1, rstd1 = torch.empty_like(some), torch.empty_like(some), torch.empty(n, device="cuda")
    wc.rms_norm_async(x, w, N, DIM, 1e-5, y_dev=y, codes_dev=codes, scales_dev=scales, residual_dev=x, sum_dev=total,
                      rstd_dev=rstd)
    wc.rms_norm_async(some, w, n, DIM, 1e-5, y_dev=y1, codes_dev=codes1, scales_dev=scales1, residual_dev=some,
                      sum_dev=total1, rstd_dev=rstd1)
    for got, want in ((total, total1), (y, y1), (codes, codes1), (scales, scales1), (rstd, rstd1)):
        assert torch.equal(got[ROWS], want)
    dh1 = torch.empty_like(some)
    dy = y   # any rows do
    dy1 = dy[ROWS].clone()
    wc.rms_norm_grad_async(dy, total, w, rstd, N, DIM, dy, None, None, 0, dsum_dev=x)
    wc.rms_norm_grad_async(dy1, total1, w, rstd1, n, DIM, dh1, None, None, 0, dsum_dev=some)
    assert torch.equal(dy[ROWS], dh1)


def _check(wc, codes, scales, w, xc, xs, x, rows, cols, tokens, out, at_rows, at_tokens):
    y = torch.empty(tokens, rows, dtype=BF16 if out == "bf16" else torch.float32, device="cuda")
    W = wc.Fp8Matrix(codes, scales, rows, cols)
    need = wc.gemm_fp8_work_bytes(W, tokens)
    work = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    wc.gemm_fp8_async(W, xc, xs, tokens, y, work, need, out=out)
    want = x @ w.t()
    assert within(y[at_tokens][:, at_rows], want, gemm_tolerance(x, w, out == "bf16", want))


def test_many_results(wc):
    rows, cols = 4200, 16
    g = torch.Generator().manual_seed(2)
    codes, scales, w = matrix_codes(torch.randn(rows, cols, generator=g))
    xc, xs = quantised(torch.randn(N, cols, generator=g))
    at = [0, (1 << 31) // rows, (1 << 32) // rows - 1, (1 << 32) // rows, N - 1]
    x = values_of(xc.view(torch.uint8)[at]) * per_column(xs[at], cols)
    log(f"case: gemm_fp8 {rows}x{cols}, {N} tokens")
    _check(wc, codes.cuda(), scales.cuda(), w, xc.cuda(), xs.cuda(), x, rows, cols, N, "bf16", slice(None), at)


@pytest.mark.parametrize("tokens,out", [(3, "f32"), (70, "f32"), (70, "bf16"), (300, "bf16")])
def test_large_matrix(wc, tokens, out):
    rows, cols = 1 << 20, 4112   # 2^32 + 2^24 codes
    g = torch.Generator().manual_seed(3)
    at = torch.tensor([0, (1 << 31) // cols, (1 << 32) // cols - 1, (1 << 32) // cols, rows - 1])
    codes = torch.randint(0, 127, (1 << 12, cols), generator=g, dtype=torch.uint8).cuda().repeat(rows >> 12, 1)
    codes[at.cuda()] = torch.randint(0, 127, (5, cols), generator=g, dtype=torch.uint8).cuda()
    scales = torch.exp2(torch.randint(-12, -8, (rows // 128, -(-cols // 128)), generator=g).float())
    w = values_of(codes[at.cuda()]) * per_column(scales[at // 128], cols)
    xc, xs = quantised(torch.randn(tokens, cols, generator=g))
    x = values_of(xc) * per_column(xs, cols)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens, {out}")
    _check(wc, codes, scales.cuda(), w, xc.cuda(), xs.cuda(), x, rows, cols, tokens, out, at.cuda(), slice(None))


@pytest.mark.parametrize("shift", [0, 1])   # whole 16 bytes, and elements one by one
def test_long_gradient(wc, shift):
    n = (1 << 32) + 5
    log(f"case: clip_grads of {n} elements, {shift} behind 16 bytes")
    g = torch.zeros(n + shift, dtype=BF16, device="cuda")[shift:]
    far = {0: 3.0, (1 << 31) + 1: 4.0, n - 1: 12.0}
    for at, v in far.items():
        g[at] = v
    norm = torch.empty(1, device="cuda")
    grads = wc.GradList([g])
    work = torch.empty(wc.clip_grads_work_bytes(grads), dtype=torch.uint8, device="cuda")
    wc.clip_grads_async(grads, 6.5, norm, work, work.numel())
    assert float(norm) == 13.0
    for at, v in far.items():
        assert float(g[at]) == v / 2
    assert int(torch.count_nonzero(g[:1 << 31])) == 1 and int(torch.count_nonzero(g[1 << 31:])) == 2
