"""GPU tests of products with e4m3 matrices on the kernels that the sizes of the other tests do not reach."""
import pytest
import torch

from e4m3_ref import UBF16, _largest_of_eights, blocks, within
from gpu_util import log
from test_gpu_gemm_fp8 import _case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


# (rows, cols, tokens, result), and the kernel that it is here for (tests/test_gemm_plan.py holds both together)
KERNELS = [
    ((4138, 400, 49, "bf16"), "32x64 bf16 once"), ((4139, 400, 64, "f32"), "32x64 f32 once"),
    ((131, 4016, 403, "bf16"), "32x64 bf16 splits"), ((133, 4048, 411, "f32"), "32x64 f32 splits"),
    ((2058, 4080, 35, "bf16"), "64x64 bf16 once splits"), ((2061, 4064, 61, "f32"), "64x64 f32 once splits"),
    ((16645, 1296, 171, "bf16"), "128x64 bf16"), ((33134, 400, 33, "bf16"), "128x64 bf16 once"),
    ((33134, 400, 61, "f32"), "128x64 f32 once"), ((4106, 4048, 33, "bf16"), "128x64 bf16 once pair splits"),
    ((4107, 4112, 62, "f32"), "128x64 f32 once pair splits"), ((261, 8240, 772, "bf16"), "128x128 bf16 splits"),
    ((883, 144, 45015, "f32"), "128x128 f32"), ((261, 656, 33100, "f32"), "128x128 f32"),
    ((32790, 400, 97, "bf16"), "256x128 bf16 once"), ((32785, 272, 128, "f32"), "256x128 f32 once"),
    ((8387, 5456, 65, "bf16"), "256x128 bf16 once splits"), ((4105, 8480, 66, "f32"), "256x128 f32 once splits"),
    ((129, 19424, 2124, "bf16"), "256x128 bf16 splits"), ((2751, 8176, 131, "f32"), "256x128 f32 splits"),
]


@pytest.mark.parametrize("size,kernel", KERNELS, ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_kernels(wc, size, kernel):
    rows, cols, tokens, out = size
    codes, scales, w, xc, xs, x = _case(rows, cols, tokens, rows)
    log(f"case: gemm_fp8 {rows}x{cols}, {tokens} tokens: {kernel}")
    W = wc.Fp8Matrix(codes.cuda(), scales.cuda(), rows, cols)
    y = _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)
    xd, wd = x.cuda(), w.cuda()
    want = xd @ wd.t()
    tol = 2.0 ** -23 * (128 + 2 * blocks(cols) + 4) * (xd.abs() @ wd.abs().t()) + 1e-40
    if out == "bf16":
        tol += 2.0 ** -11 * _largest_of_eights(x, w).cuda()
        tol += UBF16 * (want.abs() + tol)
    assert within(y, want.cpu(), tol.cpu())
    assert torch.equal(y, _run(wc, W, xc.cuda(), xs.cuda(), tokens, out)), "two runs differ"
