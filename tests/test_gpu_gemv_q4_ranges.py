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


# From 8192 rows on, 1 and 2 vectors take 4 waves per workgroup (8 below), and 3 and more 32 rows (16 below), of 8 waves
# from 5 on (they are rounded up to 4, 8 or 16 vectors).  The last workgroup has 1, 17, 31 or all of its rows.
TALL = [(8192, 128, 128, False), (8193, 1152, 32, True), (8209, 1152, 32, False), (8193, 1000, 64, True),
        (8209, 1160, 96, False), (8209, 1024, 64, True), (8223, 512, 65536, True), (8193, 2048, 128, False),
        (8192, 104, 32, True), (8209, 640, 128, True), (8193, 576, 96, True), (8209, 512, 64, False)]


@pytest.mark.parametrize("rows,cols,group,zeros", TALL)
def test_tall_matrices(wc, rows, cols, group, zeros):
    codes, scales, z, w = q4_case(rows, cols, group, zeros, rows + cols)
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    for vecs in (1, 2, 3, 4, 5, 8, 9, 16):
        x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(cols + vecs)).to(BF16)
        log(f"case: gemv_q4 {rows}x{cols} group {group} zeros {zeros} vecs {vecs}")
        y = _run(wc, matrix, x.cuda())
        assert within(y, x.double() @ w.t(), q4_tolerance(w, x.double())), vecs
        again = _run(wc, matrix, x.cuda())
        assert torch.equal(y.view(torch.int32), again.view(torch.int32)), "two runs differ"
        if group == 32 and cols % 128 == 0:     # scales and zero points off their alignment: another kernel, the same bits
            groups = cols // group
            shifted = torch.empty(rows * groups + 1, dtype=BF16, device="cuda")[1:].reshape(rows, groups)
            shifted.copy_(scales)
            other = wc.Q4Matrix(codes, shifted, rows, cols, group, zeros=z)
            assert torch.equal(_run(wc, other, x.cuda()).view(torch.int32), y.view(torch.int32)), vecs


@pytest.mark.parametrize("vecs", [1, 3, 8, 16])
def test_tall_matrices_with_values_that_are_not_finite(wc, vecs):
    """An infinity in one vector and a NaN in another reach no other vector, and no row that has a zero weight there
    gets anything but NaN for it."""
    rows, cols, group = 8209, 384, 64
    codes, scales, z, w = q4_case(rows, cols, group, True, 1)
    matrix = wc.Q4Matrix(codes, scales, rows, cols, group, zeros=z)
    x = torch.randn(vecs, cols, generator=torch.Generator().manual_seed(9)).to(BF16)
    x[0, 70] = float("inf")
    if vecs > 2:
        x[2, 383] = float("nan")
    log(f"case: gemv_q4 {rows}x{cols} vecs {vecs}, not finite")
    y = _run(wc, matrix, x.cuda()).cpu().double()
    ref = torch.stack([(w * v).sum(dim=1) for v in x.double()])
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(y[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
    tol = q4_tolerance(w, torch.nan_to_num(x.double(), 0.0, 0.0, 0.0))
    assert bool(((y - ref).abs()[fin] <= tol[fin]).all())
