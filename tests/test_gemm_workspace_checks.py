"""The workspace that products with e4m3 matrices ask for, on the CPU: a call that needs one is refused without it, with one
that is misaligned, and with one that is too short, before any launch."""
import ctypes

import pytest

P = 1 << 24
INV = -1


@pytest.fixture(scope="module")
def wc():
    from lossless_entropy_coded_amd import wc as mod
    return mod


@pytest.mark.parametrize("kind", [0, 1])                   # fp32 and bf16 results
@pytest.mark.parametrize("rows,cols,tokens", [(4096, 1 << 16, 33), (4096, 1 << 16, 64), (130, 16400, 300),
                                              (1001, 4112, 333), (1024, 14336, 100)])
def test_workspace_refusals(wc, rows, cols, tokens, kind):
    lib, W, b = wc._lib, ctypes.byref(wc._Fp8(P, P, rows, cols)), ctypes.c_uint64(0)
    assert lib.wc_gemm_fp8_work_bytes(W, tokens, ctypes.byref(b)) == wc.WC_OK
    assert b.value >= 2 * 4 * rows * tokens, "these sizes are summed in splits, two at least"
    for work, size in ((0, b.value), (P + 128, b.value), (P + 4, b.value), (P, b.value - 1), (P, 0), (0, 0)):
        assert lib.wc_gemm_fp8_async(W, P, P, tokens, P, kind, work, size, None) == INV, (work - P, size)
