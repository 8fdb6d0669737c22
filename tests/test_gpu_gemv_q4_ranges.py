"""GPU tests of the 4-bit products with scales and vectors of any finite size, and of matrices that take 32 rows per
workgroup or 4 waves."""
import pytest
import torch

from gpu_util import log
from operator_ref import q4_case, q4_tolerance, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _run(wc, matrix, x):
    vecs, rows = x.shape[0], matrix.rows
    y = torch.full((vecs * rows + 64,), float("nan"), device="cuda")
    wc.gemv_q4_async(matrix, x, vecs, y)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[vecs * rows:]).all()), "wrote past y"
    return y[:vecs * rows].reshape(vecs, rows)


def _scaled(scales, w, group, power):
    """Scales times 2^power (a number, or one per row), rounded to bf16, and the matrix in 64 bits that goes with them."""
    new = (scales.float() * torch.exp2(torch.as_tensor(power, dtype=torch.float32)).cuda()).to(BF16)
    at = torch.arange(w.shape[1]) // group
    return new, w / scales.cpu().double()[:, at] * new.cpu().double()[:, at]


@pytest.mark.parametrize("vecs", [1, 2, 3, 8, 16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("scale,size", [(106, -60), (120, -120), (126, -70), (100, -126), (-120, 110), (-126, 120),
                                        (-60, 100), (60, -100), (0, 0)])
def test_scales_of_any_size(wc, group, vecs, scale, size):
    """Scales of about 2^scale (subnormal ones too) with x of about 2^size: no sum on the way overflows or is lost where
    the result is in range.  (The products are within fp32's range, so the tolerance's steps are relative to them.)"""
    rows, cols = 40, 1024
    codes, scales, z, w = q4_case(rows, cols, group, True, group + vecs)
    scales, w = _scaled(scales, w, group, scale)
    x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(vecs)) * 2.0 ** size
    x = x.to(BF16)
    x64 = x.double()
    log(f"case: gemv_q4 scales 2^{scale}, x 2^{size}, group {group}, vecs {vecs}")
    y = _run(wc, wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z), x.cuda())
    assert within(y, x64 @ w.t(), q4_tolerance(w, x64))


@pytest.mark.parametrize("vecs", [1, 5])
def test_scales_of_different_size(wc, vecs):
    """Rows with scales from 2^-120 to 2^120 side by side, vectors from 2^-120 to 2^120 too: every result in range is
    within its own tolerance (those beyond it are infinite, or NaN
    where partial sums are infinite either way)."""
    rows, cols, group = 64, 512, 64
    codes, scales, z, w = q4_case(rows, cols, group, True, 7)
    power = torch.linspace(-120, 120, rows).round()
    scales, w = _scaled(scales, w, group, power[:, None])
    x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(3))
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    for size in (-120, -60, 0, 60, 110):
        xs = (x * 2.0 ** size).to(BF16)
        log(f"case: gemv_q4 scales from 2^-120 to 2^120, x 2^{size}, vecs {vecs}")
        y = _run(wc, matrix, xs.cuda()).cpu().double()
        ref, x64 = xs.double() @ w.t(), xs.double()
        bound = x64.abs() @ w.abs().t()
        # a product below 2^-126 is rounded to a multiple of 2^-149, each of the 2 cols steps by half of one at most
        tol = q4_tolerance(w, x64) + cols * 2.0 ** -149
        fits = bound < 2.0 ** 127
        assert bool(((y - ref).abs() <= tol)[fits].all()), size
        gone = (ref.abs() > 2.0 ** 129)
        assert not bool(torch.isfinite(y[gone]).any()), size
