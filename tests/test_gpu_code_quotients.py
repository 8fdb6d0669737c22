"""GPU tests that e4m3 codes are what their definition says, bit for bit: scale = max(largest, 2^-100) * (1 / 448) and
code = y / scale, each rounded to fp32 (1 / 448 too), the code then to e4m3."""
import pytest
import torch

from e4m3_ref import BLOCK, VALUES, block_max, blocks, per_column
from gpu_util import log

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
MANTISSAS = 1.0 + torch.arange(128, dtype=torch.float64) / 128


@pytest.fixture(scope="module")
def wc():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from lossless_entropy_coded_amd import wc as mod
    return mod


def _rounded(q):
    """Codes (bytes) of fp32 quotients in 64 bits: the nearest value, of two as near the one whose mantissa is even."""
    grid = VALUES[:127]
    top = torch.bucketize(q.abs(), grid).clamp(1, 126)
    lower, upper = q.abs() - grid[top - 1], grid[top] - q.abs()
    code = torch.where((upper < lower) | ((upper == lower) & (top % 2 == 0)), top, top - 1)
    return (code + torch.where(torch.signbit(q), 128, 0)).to(torch.uint8)


def _definition(y):
    """Codes and scales of fp32 values; a quotient in 64 bits and then in 32 is rounded as one in 32 is (53 bits are more
    than twice 24 and 2)."""
    assert y.dtype in (torch.float32, BF16)
    y = y.double()
    scales = block_max(y).clamp_min(2.0 ** -100).float() * torch.tensor(1 / 448, dtype=torch.float32)
    return _rounded((y / per_column(scales, y.shape[1])).float().double()), scales


def _check(codes, scales, y):
    want, want_scales = _definition(y)
    assert torch.equal(scales.cpu(), want_scales)
    differ = codes.cpu().view(torch.uint8) != want
    assert not bool(differ.any()), (f"{int(differ.sum())} of {differ.numel()} codes, the first of "
                                    f"{float(y[differ][0]):.9g}")


@pytest.mark.parametrize("size", [-99, -41, -40, -39, 0, 100, 126])
def test_every_pair_of_mantissas(wc, size):
    """Every mantissa that bf16 has as a block's largest value, over every mantissa at every distance that has a code, of
    both signs; zeros keep theirs."""
    small = (MANTISSAS[:, None] * torch.exp2(-torch.arange(19, dtype=torch.float64))).flatten()
    rows = []
    for top in MANTISSAS:
        y = small[small <= top]
        y = torch.cat((y, -y, torch.tensor([0.0, -0.0], dtype=torch.float64)))
        y = torch.nn.functional.pad(y, (0, -len(y) % (BLOCK - 1))).reshape(-1, BLOCK - 1)
        rows.append(torch.cat((top.expand(len(y), 1), y), dim=1))
    x = (torch.cat(rows) * 2.0 ** size).to(BF16)
    n = x.shape[0]
    codes, scales = torch.empty(n, BLOCK, dtype=torch.uint8, device="cuda"), torch.empty(n, 1, device="cuda")
    log(f"case: quant_fp8 of every pair of mantissas, 2^{size}")
    wc.quant_fp8_async(x.cuda(), n, BLOCK, codes, scales)
    _check(codes, scales, x.float())


@pytest.mark.parametrize("n,dim,size", [(64, 4096, 1.0), (9, 8200, 1.0), (300, 136, 1.0), (64, 4096, 2.0 ** -60),
                                        (64, 1024, 2.0 ** -120)])
def test_norm_into_codes(wc, n, dim, size):
    """The norm's y in fp32 is h * rstd * weight, product by product, of the rstd that it returns: its codes are those."""
    g = torch.Generator().manual_seed(dim)
    x, w = torch.randn(n, dim, generator=g).to(BF16), (torch.randn(dim, generator=g) * size).to(BF16)
    codes, scales = torch.empty(n, dim, dtype=torch.uint8, device="cuda"), torch.empty(n, blocks(dim), device="cuda")
    rstd = torch.empty(n, device="cuda")
    log(f"case: rms_norm into codes, {n}x{dim}, weights of {size:g}")
    wc.rms_norm_async(x.cuda(), w.cuda(), n, dim, 1e-5, codes_dev=codes, scales_dev=scales, rstd_dev=rstd)
    _check(codes, scales, x.float() * rstd.cpu()[:, None] * w.float())
