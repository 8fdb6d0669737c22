"""GPU tests of clipping where the quotient of the bound and the norm is below fp32's normal range, and the results are not."""
import math

import pytest
import torch

from e4m3_ref import UBF16, within
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1])                                   # whole 16 bytes, and elements one by one
@pytest.mark.parametrize("size,bound", [(1e37, 1.0), (1e37, 1e-3), (1e36, 1e-20), (1e37, 1e-35), (1e30, 1e-9), (1e-30, 1e-33)])
def test_small_quotients(wc, size, bound, shift, kind):
    g = torch.Generator().manual_seed(2)
    log(f"case: clip_grads of {size:g} to {bound:g} {kind} {shift}")
    grads = [(torch.randn(n + shift, generator=g).clamp(-3, 3) * (size / 8)).to(kind).cuda()[shift:] for n in (9, 50)]
    outs = [torch.empty_like(t) for t in grads]
    handle, norm = wc.GradList(grads, outs), torch.empty(1, device="cuda")
    work = torch.empty(wc.clip_grads_work_bytes(handle), dtype=torch.uint8, device="cuda")
    wc.clip_grads_async(handle, bound, norm, work, work.numel())
    want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    assert bound < want < 3e38 and math.isfinite(float(norm))
    for t, out in zip(grads, outs):
        exact = t.cpu().double() * (float(torch.tensor(bound)) / want)
        # the factor is rounded and the product, each by half a step; results below the normal range by two of theirs
        tol = (2.0 ** -23 + 1e-12) * exact.abs() + 2.0 ** -148
        assert within(out, exact, tol + (UBF16 * (exact.abs() + tol) + 2.0 ** -134 if kind == BF16 else 0.0))
