"""GPU tests of which products the sums of e4m3 products keep: all, but in bf16 results of more than 32 tokens."""
import pytest
import torch

from cancelling import cancelling, codes_of
from e4m3_ref import UBF16, blocks, gemm_tolerance, within
from gpu_util import log
from test_gpu_gemm_fp8 import _case, _run

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


FEW = [(1, 16, 1), (17, 144, 3), (129, 256, 17), (100, 1168, 5), (1024, 4096, 1), (2000, 272, 32), (96, 65536, 3),
       (4096, 400, 3), (4097, 1168, 16), (4100, 272, 17), (8209, 4112, 31), (10240, 400, 5), (16384, 272, 1), (16385, 272, 16)]


@pytest.mark.parametrize("rows,cols,tokens", FEW)
def test_few_tokens_in_bf16(wc, rows, cols, tokens):
    """bf16 results of up to 32 tokens are fp32 sums of every product, rounded once: no allowance for dropped ones."""
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, rows + tokens)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens, bf16, every product")
    y = _run(wc, wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols), xc.cuda(), xs.cuda(), tokens, "bf16")
    want = x @ w.t()
    tol = gemm_tolerance(x, w, False, want)
    assert within(y, want, tol + UBF16 * (want.abs() + tol))


@pytest.mark.parametrize("rows,cols,tokens,out", [
    (200, 256, 1, "f32"), (200, 1296, 20, "f32"), (300, 2096, 60, "f32"), (1003, 2096, 333, "f32"), (130, 16400, 300, "f32"),
    (2751, 8176, 131, "f32"), (261, 656, 33100, "f32"), (200, 256, 1, "bf16"), (200, 1296, 20, "bf16"), (4100, 400, 16, "bf16"),
    (4100, 272, 32, "bf16"), (10250, 400, 9, "bf16")])
def test_products_beside_larger_ones(wc, rows, cols, tokens, out):
    """Products that 8-bit instructions drop, 2^16 below the largest of their eight, beside large ones that cancel: fp32
    results, and those of up to 32 tokens, are what whole numbers give."""
    codes, xc, want = cancelling(rows, cols, tokens)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens, {out}, products beside larger ones")
    ones = torch.ones(blocks(rows) * blocks(cols), device="cuda")
    W = wc.Fp8Matrix(codes_of(codes).cuda(), ones, rows, cols)
    y = _run(wc, W, codes_of(xc).cuda(), torch.ones(tokens, blocks(cols), device="cuda"), tokens, out)
    assert torch.equal(y.cpu().double(), want.to(BF16).double() if out == "bf16" else want)
